// Attention over grouped heads: O = softmax(scale * Q K^T, over the allowed keys) V.
//
// Row r of a kv head's problem is query token r / G of its q head r % G (G q heads share a kv head), so
// the heads of a group read each key and value once, also where there is one query token.  Keys go by
// in tiles, with the running maximum m and sum l of the softmax per row (one pass):
//     p = exp2(c s - c m),  l += sum p,  O += p v,      c = scale * log2(e);
// where m moves, l and O are multiplied by exp2(c m_old - c m_new).
//
// The products are computed transposed, S^T = K Q^T and O^T = V^T P^T, with 16x16x32 MFMAs: a lane then
// holds scores of one query (lane (q, l16) of a 16x16 block: query l16, keys 4q .. 4q + 3), the factors of m
// and l are one number per lane, and the probabilities, rounded to bf16 in pairs, are already
// the B operand of the second product: its K order is the order in which the lane holds them (keys 4q ..
// of one 16-key block, then of the next), and V^T is read from LDS in that order by transposing reads.
// 16x16x32 and not 32x32x16: on this SIMD a 16x16x32 MFMA leaves room for two vector instructions, a
// 32x32x16 one (2x the work) for none, and the exponentials are as long as the products.
//
// Vector instructions per score are what is saved on:
//   * l is a matrix product too (P^T with ones), which also makes it the sum of the rounded probabilities;
//   * m is not followed tile by tile.  It stays where it was, kHeadroom powers of two above the largest score
//     then seen (fp32 and bf16 have the exponents for it), as long as every new p is below 2, which one
//     OR over the packed probabilities tells (bit 14 of a positive bf16 is set from 2 on); only
//     otherwise is the maximum taken, O and l rescaled and the probabilities computed again.
// The exponents c s - c m are one fused operation each, exact before its one rounding.  Past kLarge the rounding of c m alone is
// worth more than the headroom, so c s is rounded too, the same way, and equal scores have equal exponents again
// (the row's other scores are then a unit of c m, 32 powers of two, or more away).
//
// Rounding to bf16: the probabilities before the second product (the matrix cores' input; relative
// 2^-8 each, averaged over the keys) and O at the store.  Scores, m, l and O are fp32.  O is kept undivided, with the
// largest p anywhere from 2^-32 to 2: values v below 2^-70 or above 2^90 in magnitude leave fp32's range there.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

// Two bf16 in one word, rounded to nearest even (one instruction).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}

constexpr float kNegInf = -__builtin_inff();
constexpr float kHeadroom = 32.f;  // powers of two between the largest score and 1; p reaches 2^33 times as much before m moves
constexpr float kLarge = 0x1p28f;  // of |c m|: its last place is worth 32 from here on
constexpr uint32_t kTooLarge = 0x40004000u;  // a packed pair of p has one of 2 or more

// ---- layouts in LDS: rows of D elements in 16-byte chunks, chunk c of row r at position c ^ swz(r) ----
// K is read 16 bytes per lane from 16 consecutive rows at one chunk, which must land in 16 different
// 16-byte bank groups of the 256-byte line (and lanes l and l + 16 in one 32-byte block: k_chunk).
template <int D>
__device__ __forceinline__ int k_swz(int r) {
    return D == 128 ? (r & 15) : ((r >> 1) & 7);
}
// V is read by transposing reads, 8 bytes per lane: 16 lanes take 4 rows x 32 bytes, half a wave 8
// consecutive rows, whose 32-byte pieces must not share banks.
template <int D>
__device__ __forceinline__ int v_swz(int r) {
    return D == 128 ? (r & 7) << 1 : ((r >> 1) & 3) << 1;
}

// One wave's state for NQ blocks of 16 rows.
template <int D, int NQ>
struct Rows {
    bf16x8_t q[D / 32][NQ];  // B operand: lane (q, query): chunk k_chunk(ks, q)
    f32x4_t o[D / 16][NQ];   // O^T: lane (q, query), columns 16 db + 4q ..
    f32x4_t l[NQ];           // the softmax's sum (four times the same)
    float mc[NQ];            // what the exponents subtract: c times the maximum then seen + kHeadroom; -inf: no key yet
};

// Scores of a tile of KB blocks of 16 keys: [key block][row block], keys 16 kb + 4q ..
template <int KB, int NQ>
struct Scores {
    f32x4_t s[KB][NQ];
};
// Their probabilities as B operands: [32-key block][row block].
template <int KB, int NQ>
struct Probs {
    u32x4_t p[KB / 2][NQ];
};

template <int D, int NQ>
__device__ __forceinline__ void rows_init(Rows<D, NQ>& w) {
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
#pragma unroll
        for (int b = 0; b < D / 16; ++b) w.o[b][qb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        w.l[qb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        w.mc[qb] = kNegInf;
    }
}

// The lane's byte offsets into a K and a V tile, without the constants that the compiler folds into the
// instructions: K row l16 at chunk k_chunk (rows 16 apart have the same swizzle), V row 4q + l16 / 4 at
// column block b (rows 16 apart as well).
template <int D>
struct Offsets {
    int k[D / 32], v[D / 16];
};

template <int D>
__device__ __forceinline__ Offsets<D> offsets() {
    const int lane = int(threadIdx.x) & 63;
    const int q = lane >> 4, l16 = lane & 15;
    Offsets<D> f;
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks) f.k[ks] = l16 * (2 * D) + ((k_chunk(ks, q) ^ k_swz<D>(l16)) << 4);
#pragma unroll
    for (int b = 0; b < D / 16; ++b) {
        const int r = 4 * q + (l16 >> 2), chunk = 2 * b + ((l16 & 3) >> 1);
        f.v[b] = r * (2 * D) + ((chunk ^ v_swz<D>(r)) << 4) + 8 * (l16 & 1);
    }
    return f;
}

// Scores of the K tile at kt.
template <int D, int NQ, int KB>
__device__ __forceinline__ void scores(const Rows<D, NQ>& w, const Offsets<D>& f, const unsigned char* kt, Scores<KB, NQ>& x) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
        for (int qb = 0; qb < NQ; ++qb) x.s[kb][qb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            const bf16x8_t k = *reinterpret_cast<const bf16x8_t*>(kt + f.k[ks] + kb * 16 * (2 * D));
#pragma unroll
            for (int qb = 0; qb < NQ; ++qb)
                x.s[kb][qb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, w.q[ks][qb], x.s[kb][qb], 0, 0, 0);
        }
    }
}

// Scores of keys that a lane's query does not take (bit of its `allowed` clear) to -inf.
template <int KB, int NQ>
__device__ __forceinline__ void mask_scores(Scores<KB, NQ>& x, const uint64_t (&allowed)[NQ]) {
    asm volatile("");  // a branch, not a select in every tile
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
        const uint64_t mine = allowed[qb] >> ((threadIdx.x & 48) >> 2);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const uint32_t bits = uint32_t(mine >> (16 * kb));
#pragma unroll
            for (int i = 0; i < 4; ++i) x.s[kb][qb][i] = (bits >> i) & 1u ? x.s[kb][qb][i] : kNegInf;
        }
    }
}

// m follows the largest of the scores where it has to, and l and O follow m.
template <int D, int NQ, int KB>
__device__ __forceinline__ void grow(Rows<D, NQ>& w, const Scores<KB, NQ>& x, float c) {
#pragma clang fp contract(off)  // c m is the rounded product, as in probabilities()
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
        float top = kNegInf;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, x.s[kb][qb][i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32)) * c;
        // p below 2: the packed test's bound, with its rounding
        const bool move = top > kNegInf && !(top - w.mc[qb] < 0.99f);
        if (__any(move)) {
            const float mc = move ? top + kHeadroom : w.mc[qb];
            const float f = move ? __builtin_amdgcn_exp2f(w.mc[qb] - mc) : 1.f;
            w.mc[qb] = mc;
#pragma unroll
            for (int i = 0; i < 4; ++i) w.l[qb][i] *= f;
#pragma unroll
            for (int b = 0; b < D / 16; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) w.o[b][qb][i] *= f;
        }
    }
}

// The probabilities of x; returns an OR of them all.  ANY: rows whose |c m| is kLarge or more among them, which subtract it
// after the product's rounding.
template <bool ANY, int D, int NQ, int KB>
__device__ __forceinline__ uint32_t probabilities(const Rows<D, NQ>& w, const Scores<KB, NQ>& x, Probs<KB, NQ>& p, float c) {
    uint32_t any = 0;
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
        const float all = w.mc[qb] == kNegInf ? 0.f : w.mc[qb];  // without a key yet every score is -inf
        const bool large = ANY && !(__builtin_fabsf(all) < kLarge);
        const float mc = large ? 0.f : all, after = large ? all : 0.f;
        auto power = [&](float s) __attribute__((always_inline)) {
            const float e = __builtin_fmaf(s, c, -mc);
            return __builtin_amdgcn_exp2f(ANY ? e - after : e);
        };
#pragma unroll
        for (int kk = 0; kk < KB / 2; ++kk)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x4_t& s = x.s[2 * kk + e / 2][qb];
                const float lo = power(s[2 * (e % 2)]);
                const float hi = power(s[2 * (e % 2) + 1]);
                const uint32_t v = pack_bf16(lo, hi);
                p.p[kk][qb][e] = v;
                any |= v;
            }
    }
    return any;
}

// O += P V for the V tile at vt, and l.
template <int D, int NQ, int KB>
__device__ __forceinline__ void weighted(Rows<D, NQ>& w, const Offsets<D>& f, const unsigned char* vt, const Probs<KB, NQ>& p) {
    const bf16x8_t ones = __builtin_bit_cast(bf16x8_t, u32x4_t{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
#pragma unroll
    for (int kk = 0; kk < KB / 2; ++kk) {  // 32 keys each
#pragma unroll
        for (int qb = 0; qb < NQ; ++qb)
            w.l[qb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, __builtin_bit_cast(bf16x8_t, p.p[kk][qb]), w.l[qb], 0, 0, 0);
#pragma unroll
        for (int b = 0; b < D / 16; ++b) {
            s16x4_t v[2];
#pragma unroll
            for (int part = 0; part < 2; ++part)
                v[part] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4_t*)(vt + f.v[b] + (32 * kk + 16 * part) * (2 * D)));
            const bf16x8_t a = __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
            for (int qb = 0; qb < NQ; ++qb)
                w.o[b][qb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, p.p[kk][qb]), w.o[b][qb], 0, 0, 0);
        }
    }
}

// The probabilities of x, to a maximum that has moved if one of them would reach 2.
template <int D, int NQ, int KB>
__device__ __forceinline__ void probabilities_checked(Rows<D, NQ>& w, const Scores<KB, NQ>& x, Probs<KB, NQ>& p, float c) {
    const uint32_t any = probabilities<false>(w, x, p, c);
    bool again = (any & kTooLarge) != 0;
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) again = again || !(__builtin_fabsf(w.mc[qb]) < kLarge);  // no key yet (-inf) among them
    if (__any(again)) {
        grow(w, x, c);
        bool large = false;
#pragma unroll
        for (int qb = 0; qb < NQ; ++qb) large = large || (w.mc[qb] != kNegInf && !(__builtin_fabsf(w.mc[qb]) < kLarge));
        if (__any(large))
            probabilities<true>(w, x, p, c);
        else
            probabilities<false>(w, x, p, c);
    }
}

// One tile's values and the next tile's scores: the exponentials of x (scores of the tile whose values are
// at vt) are taken while the matrix cores compute xn, the scores of the K tile at kt.
template <int D, int NQ, int KB>
__device__ __forceinline__ void fused_step(Rows<D, NQ>& w, const Offsets<D>& f, const unsigned char* kt, const unsigned char* vt,
                                           const Scores<KB, NQ>& x, Scores<KB, NQ>& xn, float c) {
    Probs<KB, NQ> p;
    scores(w, f, kt, xn);
    probabilities_checked(w, x, p, c);
    weighted(w, f, vt, p);
}

__device__ __forceinline__ bool pair_finite(uint32_t v) { return (v & 0x7F80u) != 0x7F80u && (v & 0x7F800000u) != 0x7F800000u; }

// Zero in a matrix product does not silence an infinity or a NaN, so tiles with keys that some query leaves
// out are looked over first.  tidy_v: rows [first, first + rows) of the V tile, one wave: rows of
// keys that nobody takes (bit of `live` clear) become zeros; says whether another row holds an infinity
// or a NaN.  CLEAN: those become zeros as well.
template <int D, bool CLEAN>
__device__ __forceinline__ bool tidy_v(unsigned char* vt, int first, int rows, uint64_t live) {
    int lane = int(threadIdx.x) & 63;
    asm volatile("" : "+v"(lane));  // addresses computed here, not held through the main loop
    bool odd = false;
    for (int i = lane; i < rows * (D / 8); i += 64) {
        const int r = first + i / (D / 8);  // any order within the row will do
        u32x4_t* at = reinterpret_cast<u32x4_t*>(vt + first * (2 * D) + i * 16);
        const bool take = (live >> r) & 1;
        u32x4_t x = *at;
        bool fine = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) fine = fine && pair_finite(x[e]);
        if (!take) {
            *at = u32x4_t{0, 0, 0, 0};
        } else if (!fine) {
            odd = true;
            if constexpr (CLEAN) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if ((x[e] & 0x7F80u) == 0x7F80u) x[e] &= 0xFFFF0000u;
                    if ((x[e] & 0x7F800000u) == 0x7F800000u) x[e] &= 0xFFFFu;
                }
                *at = x;
            }
        }
    }
    return odd;
}

// The infinities and NaN of a V tile, before tidy_v cleans them away, added to the queries that take their
// keys: what a positive probability times an infinity or a NaN gives is that infinity or NaN.
template <int D, int NQ>
__device__ __forceinline__ void add_nonfinite(Rows<D, NQ>& w, const unsigned char* vt, int keys, const uint64_t (&allowed)[NQ]) {
    int q = (int(threadIdx.x) >> 4) & 3;
    asm volatile("" : "+v"(q));
    for (int j = 0; j < keys; ++j) {
        bool mine[NQ], some = false;
#pragma unroll
        for (int qb = 0; qb < NQ; ++qb) {
            mine[qb] = (allowed[qb] >> j) & 1;
            some = some || mine[qb];
        }
        if (!__any(some)) continue;
#pragma unroll
        for (int b = 0; b < D / 16; ++b) {  // columns 16 b + 4 q ..
            const u32x2_t v = *reinterpret_cast<const u32x2_t*>(
                vt + j * (2 * D) + (((2 * b + (q >> 1)) ^ v_swz<D>(j)) << 4) + 8 * (q & 1));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t bits = i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16;
                const bool odd = (bits & 0x7F800000u) == 0x7F800000u;
#pragma unroll
                for (int qb = 0; qb < NQ; ++qb)
                    if (mine[qb] && odd) w.o[b][qb][i] += __uint_as_float(bits);
            }
        }
    }
}

// The Q operands of rows row0 + 16 qb + l16 (rows past the last read as zeros).
template <int D, int NQ>
__device__ __forceinline__ void load_q(Rows<D, NQ>& w, const AttnArgs& a, int b, int hk, int row0) {
    const int lane = int(threadIdx.x) & 63, q = lane >> 4;
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
        const int row = row0 + 16 * qb + (lane & 15);
        const bool in = row < a.rows;
        const int t = in ? row / a.group : 0, g = in ? row - t * a.group : 0;
        const uint16_t* src = a.q + int64_t(b) * a.q_batch + int64_t(t) * a.q_token + int64_t(hk * a.group + g) * a.q_head;
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            u32x4_t v = {0, 0, 0, 0};
            if (in) v = *reinterpret_cast<const u32x4_t*>(src + 8 * k_chunk(ks, q));
            w.q[ks][qb] = __builtin_bit_cast(bf16x8_t, v);
        }
    }
}

// O of the rows to memory, divided by l: 16 bytes per lane and pair of column blocks after an exchange between
// neighbouring lane quarters (each holds 4 of every 16 columns).  A row without keys has l = 0: zeros.
template <int D, int NQ>
__device__ __forceinline__ void store_o(const Rows<D, NQ>& w, const AttnArgs& a, int b, int hk, int row0) {
    const int lane = int(threadIdx.x) & 63, q = lane >> 4;
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
        const int row = row0 + 16 * qb + (lane & 15);
        const bool in = row < a.rows;
        const int t = in ? row / a.group : 0, g = in ? row - t * a.group : 0;
        uint16_t* dst = a.o + int64_t(b) * a.o_batch + int64_t(t) * a.o_token + int64_t(hk * a.group + g) * a.o_head;
        const float l = w.l[qb][0], f = l == 0.f ? 0.f : 1.f / l;
        auto pair = [&](float x, float y) { return pack_bf16(x * f, y * f); };
#pragma unroll
        for (int d = 0; d < D / 16; d += 2) {
            const f32x4_t x = w.o[d][qb], y = w.o[d + 1][qb];
            const auto s0 = __builtin_amdgcn_permlane16_swap(pair(x[0], x[1]), pair(y[0], y[1]), false, false);
            const auto s1 = __builtin_amdgcn_permlane16_swap(pair(x[2], x[3]), pair(y[2], y[3]), false, false);
            if (in) *reinterpret_cast<u32x4_t*>(dst + 16 * (d + (q & 1)) + 8 * (q >> 1)) = u32x4_t{s0[0], s1[0], s0[1], s1[1]};
        }
    }
}

// Partial results of the rows for the join: O unnormalised, then (c m, l).
template <int D>
__device__ __forceinline__ void store_part(const Rows<D, 2>& w, const AttnArgs& a, int64_t base, int row0) {
    const int lane = int(threadIdx.x) & 63, q = lane >> 4;
#pragma unroll
    for (int qb = 0; qb < 2; ++qb) {
        const int row = row0 + 16 * qb + (lane & 15);
        if (row >= a.rows) continue;
        float* dst = a.part + (base + row) * D;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4_t*>(dst + 16 * d + 4 * q) = w.o[d][qb];
        if (q == 0) {
            a.part_ml[2 * (base + row)] = w.mc[qb];
            a.part_ml[2 * (base + row) + 1] = w.l[qb][0];
        }
    }
}

// Keeps a wave-uniform value in a scalar register: without it the compiler reloads kernel arguments inside
// the loop, and a scalar load shares its wait with every LDS read in flight.
template <class T>
__device__ __forceinline__ T in_sgpr(T v) {
    if constexpr (sizeof(T) == 8) {
        const uint64_t x = __builtin_bit_cast(uint64_t, v);
        uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(x)), hi = __builtin_amdgcn_readfirstlane(uint32_t(x >> 32));
        asm volatile("" : "+s"(lo), "+s"(hi));
        return __builtin_bit_cast(T, (uint64_t(hi) << 32) | lo);
    } else {
        uint32_t x = __builtin_amdgcn_readfirstlane(__builtin_bit_cast(uint32_t, v));
        asm volatile("" : "+s"(x));
        return __builtin_bit_cast(T, x);
    }
}

// Workgroup barrier after LDS reads and writes that leaves copies in flight (__syncthreads() waits for them).
__device__ __forceinline__ void lds_writes_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0); vmcnt and expcnt left alone
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Keys [0, n) that a batch entry holds at all.
__device__ __forceinline__ int live_keys(const AttnArgs& a, int b) {
    int n = a.kv_len;
    if (a.lens != nullptr) {
        const int v = a.lens[b];
        n = v < 0 ? 0 : v < n ? v : n;
    }
    return n;
}

// Bits 0 .. rel (none for rel < 0).
__device__ __forceinline__ uint64_t up_to(int64_t rel) {
    return rel < 0 ? 0ull : rel >= 63 ? ~0ull : (2ull << rel) - 1;
}

// Many rows: a workgroup of 4 waves takes 64 NQ rows of one kv head, a wave 16 NQ of them; tiles of 64 keys go
// through LDS, double-buffered, by direct copies one tile ahead.  4608 x 4608, 24 heads of 128: 262 to 273 us = 956 to 996 TFLOP/s
// on different cards, of which 864 workgroups in 512 places (two rounds for 1.7) are the largest loss: 16 heads, 4096 x 16384, an exact
// round, run at 1121 TFLOP/s.  There the matrix cores are busy for 53% of the SIMD cycles at least and vector
// instructions (matrix ones' issue included) active for 45% (profiles/block_operators_kernel_trace_and_counters.txt):
// two waves per SIMD do not keep either full.  Power takes 6% and 11%: with zeros for inputs, the same instructions, 250 for
// 267 us and 433 for 490.  Heads of 64 have half the products per exponential: 4608 x 4608, 24
// heads: 161 us = 811 TFLOP/s.
template <int D, int NQ>
__global__ __launch_bounds__(256, D == 64 && NQ == 1 ? 4 : 2) void attention_kernel(AttnArgs a) {
    constexpr int kRows = 64 * NQ;                // of a workgroup
    constexpr int kTile = 64 * D * 2;
    constexpr int kRowsPerCopy = 512 / D;         // rows that one wave-wide 16-byte copy brings
    constexpr int kCopies = 64 / kRowsPerCopy / 4;  // copies per wave and tile
    // an array per buffer, not one indexed by parity: the compiler then sees that a tile's reads do not
    // depend on the copies still landing in the other buffer
    __shared__ __attribute__((aligned(1024))) unsigned char kbuf0[kTile], kbuf1[kTile], vbuf0[kTile], vbuf1[kTile];
    __shared__ int odd_tile;  // the last tile in which an infinity or a NaN was seen
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    // tiles of one head next to each other, heads of one XCD together; causal: those with the most keys first (4608
    // tokens, 24 heads of 128: 163 us, last 191)
    int id = xcd_remap(int(blockIdx.x), int(gridDim.x));
    const int rt = a.causal ? a.row_tiles - 1 - id % a.row_tiles : id % a.row_tiles;
    id /= a.row_tiles;
    const int split = id % a.splits;
    id /= a.splits;
    const int hk = id % a.kv_heads, b = id / a.kv_heads;

    const int n = in_sgpr(live_keys(a, b));
    const int row0 = rt * kRows + wave * (16 * NQ);  // the wave's rows
    const int64_t start = a.causal ? (a.start != nullptr ? a.start[b] : 0) : 0;
    // the last key of the workgroup's rows
    const int last_row = rt * kRows + kRows - 1 < a.rows ? rt * kRows + kRows - 1 : a.rows - 1;
    const int64_t last = a.causal ? start + last_row / a.group : int64_t(n) - 1;
    // the first key that a row of the workgroup leaves out by the causal rule (all rows take those before)
    const int64_t first64 = a.causal ? start + (rt * kRows) / a.group + 1 : n;
    const int64_t end64 = last + 1 < n ? last + 1 : n;
    const int end = end64 < 0 ? 0 : int(end64);
    const int first = in_sgpr(first64 < 0 ? 0 : first64 < n ? int(first64) : n);
    const int tiles = (end + 63) / 64;
    // the splits share the keys there are, not the keys there could be
    int share = tiles;
    if constexpr (NQ == 2) {  // 64 rows are taken unsplit only
        if (a.splits > 1) share = int(uint32_t(tiles + a.splits - 1) / uint32_t(a.splits));
    }
    const int t0 = split * share;
    const int t1 = in_sgpr(t0 + share < tiles ? t0 + share : tiles);

    Rows<D, NQ> w;
    rows_init(w);
    load_q(w, a, b, hk, row0);
    // the last key of the lane's rows
    int64_t mine[NQ];
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
        const int row = row0 + 16 * qb + (lane & 15);
        mine[qb] = a.causal ? start + (row < a.rows ? row : a.rows - 1) / a.group : int64_t(1) << 40;
    }
    const Offsets<D> f = offsets<D>();

    // the next tile to copy, and its key and value rows
    const uint32_t k_row = in_sgpr(uint32_t(a.k_token) * 2u), v_row = in_sgpr(uint32_t(a.v_token) * 2u);
    const unsigned char* kp = reinterpret_cast<const unsigned char*>(a.k + int64_t(b) * a.k_batch + int64_t(hk) * a.k_head) + int64_t(64) * t0 * k_row;
    const unsigned char* vp = reinterpret_cast<const unsigned char*>(a.v + int64_t(b) * a.v_batch + int64_t(hk) * a.v_head) + int64_t(64) * t0 * v_row;
    const uint8_t* mask = in_sgpr(a.mask == nullptr ? nullptr : a.mask + int64_t(b) * a.mask_batch);
    const float c = in_sgpr(a.scale_log2);
    uint32_t koff[kCopies], voff[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int r = (wave * kCopies + i) * kRowsPerCopy + lane / (D / 8), p = lane % (D / 8);
        koff[i] = uint32_t(r) * k_row + uint32_t(p ^ k_swz<D>(r)) * 16u;
        voff[i] = uint32_t(r) * v_row + uint32_t(p ^ v_swz<D>(r)) * 16u;
    }
    // The tiles' copies, each K and V tile issued once, in order.
    int k_next = t0, v_next = t0;
    auto issue_k = [&](int t, unsigned char* kd) __attribute__((always_inline)) {
        if (k_next != t || t >= t1) return;
        ++k_next;
        const uint32_t rest = uint32_t(n - 64 * t < 64 ? n - 64 * t : 64) - 1u;  // rows past the last key come as zeros
        const auto kr = make_rsrc(kp, rest * k_row + 2u * D);
        kp += uint64_t(64) * k_row;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) dma16(kr, kd + (wave * kCopies + i) * 1024, koff[i], 0);
    };
    auto issue_v = [&](int t, unsigned char* vd) __attribute__((always_inline)) {
        if (v_next != t || t >= t1) return;
        ++v_next;
        const uint32_t rest = uint32_t(n - 64 * t < 64 ? n - 64 * t : 64) - 1u;
        const auto vr = make_rsrc(vp, rest * v_row + 2u * D);
        vp += uint64_t(64) * v_row;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) dma16(vr, vd + (wave * kCopies + i) * 1024, voff[i], 0);
    };
    // Every copy issued so far is there, and every wave is done with the tiles before.
    auto arrive = [&]() __attribute__((always_inline)) {
        wait_vmcnt<0>();
        __syncthreads();
    };
    // The lane's bytes of the mask for tiles t, t + 1 and t + 2, fetched before they are needed (0 past the last key).
    auto fetch = [&](int t) __attribute__((always_inline)) {
        if (mask == nullptr) return uint8_t(0);
        return uint8_t(__builtin_amdgcn_raw_buffer_load_b8(make_rsrc(mask, uint32_t(n)), uint32_t(64 * t + lane), 0, 0));
    };
    uint8_t m0 = fetch(t0), m1 = fetch(t0 + 1), m2 = fetch(t0 + 2);
    // Whole tiles: all rows of the workgroup take all 64 keys.
    const int whole_end = in_sgpr((first < 64 * t1 ? first : 64 * t1) / 64);
    auto whole = [&](int t, uint8_t byte) __attribute__((always_inline)) {
        return t < whole_end && (mask == nullptr || __ballot(byte != 0) == ~0ull);
    };
    if (threadIdx.x == 0) odd_tile = -1;
    int t = t0;

    // One tile of any kind, in (kc, vc); the next one goes to (kn, vn).
    auto any_step = [&](unsigned char* kc, unsigned char* vc, unsigned char* kn, unsigned char* vn)
                        __attribute__((always_inline)) {
        arrive();
        const uint64_t in = n - 64 * t >= 64 ? ~0ull : (1ull << (n - 64 * t)) - 1;
        const uint64_t live = mask != nullptr ? __ballot(m0 != 0) : in;
        const bool partial = !whole(t, m0);
        m0 = m1;
        m1 = m2;
        m2 = fetch(t + 3);
        issue_k(t + 1, kn);
        issue_v(t + 1, vn);
        ++t;
        if (live == 0) return;  // the same in every wave
        uint64_t allowed[NQ];
#pragma unroll
        for (int qb = 0; qb < NQ; ++qb) allowed[qb] = ~0ull;
        bool odd = false;
        if (partial) {
#pragma unroll
            for (int qb = 0; qb < NQ; ++qb) allowed[qb] = live & up_to(mine[qb] - 64 * int64_t(t - 1));
            if (tidy_v<D, false>(vc, wave * 16, 16, live)) odd_tile = t;
            lds_writes_barrier();
            odd = odd_tile == t;
        }
        Scores<4, NQ> s;
        Probs<4, NQ> p;
        scores(w, f, kc, s);
        if (partial) mask_scores(s, allowed);
        probabilities_checked(w, s, p, c);
        if (odd) {
            add_nonfinite<D>(w, vc, 64, allowed);
            lds_writes_barrier();
            tidy_v<D, true>(vc, wave * 16, 16, live);
            lds_writes_barrier();
        }
        weighted(w, f, vc, p);
    };

    issue_k(t0, kbuf0);
    issue_v(t0, vbuf0);
    while (t < t1) {
        if (whole(t, m0) && whole(t + 1, m1) && whole(t + 2, m2)) {
            // a run of whole tiles, two per turn; the scores are one tile ahead of the values
            arrive();
            issue_k(t + 1, kbuf1);
            Scores<4, NQ> s0, s1;
            scores(w, f, kbuf0, s0);
            do {
                arrive();
                issue_k(t + 2, kbuf0);
                issue_v(t + 1, vbuf1);
                fused_step(w, f, kbuf1, vbuf0, s0, s1, c);
                arrive();
                issue_k(t + 3, kbuf1);
                issue_v(t + 2, vbuf0);
                m0 = m2;
                m1 = fetch(t + 3);
                m2 = fetch(t + 4);
                fused_step(w, f, kbuf0, vbuf1, s1, s0, c);
                t += 2;
            } while (whole(t + 1, m1) && whole(t + 2, m2));
            arrive();
            issue_v(t + 1, vbuf1);
            Probs<4, NQ> p;
            probabilities_checked(w, s0, p, c);
            weighted(w, f, vbuf0, p);
            m0 = m1;
            m1 = m2;
            m2 = fetch(t + 3);
            ++t;
        } else {
            any_step(kbuf0, vbuf0, kbuf1, vbuf1);
        }
        if (t < t1) any_step(kbuf1, vbuf1, kbuf0, vbuf0);
    }
    if constexpr (NQ == 2) {  // 64 rows are taken unsplit only
        if (a.splits > 1) {
            store_part(w, a, ((int64_t(b) * a.kv_heads + hk) * a.splits + split) * a.rows, row0);
            return;
        }
    }
    store_o(w, a, b, hk, row0);
}

// Few rows (one or two blocks of 16: decoded tokens): bound by reading the keys and values once.  Every
// wave takes its own tiles of 32 keys (tile w, w + 4, .. of the workgroup's range for wave w), copied into its own part of
// LDS, so no barrier stands between the copies; two workgroups share a compute unit, and while one wave
// computes the others' copies are on their way (up to 128 KB per compute unit).  Measured: 1 x 40007 keys, 32 / 8 heads of
// 128: 36 us = 4.5 TB/s (31 us and 5.3 TB/s in the kernel); 4 x 4099 keys: 17 us.  The waves' results are joined through LDS;
// where the keys are also split across workgroups, each leaves its partial result in the workspace and the last one to arrive joins them.  Both joins go in a fixed
// order (wave 0 .., split 0 ..), so results do not depend on timing.
constexpr int kShortKeys = 32;

template <int D, int NQ>
__global__ __launch_bounds__(256, 2) void attention_short_kernel(AttnArgs a) {
    constexpr int kTile = kShortKeys * D * 2;
    constexpr int kRowsPerCopy = 512 / D;
    constexpr int kCopies = kShortKeys / kRowsPerCopy;  // of K and of V, per wave and tile
    constexpr int kWaves = 4;
    __shared__ __attribute__((aligned(1024))) unsigned char tiles_lds[kWaves][2 * kTile];  // K, then V
    __shared__ float join_mc[kWaves][NQ][16], join_l[kWaves][NQ][16];
    __shared__ int last_split;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int q = lane >> 4, l16 = lane & 15;
    // row tiles and splits of one head next to each other on one XCD
    int id = xcd_remap(int(blockIdx.x), int(gridDim.x));
    const int split = id % a.splits;
    id /= a.splits;
    const int rt = id % a.row_tiles;
    id /= a.row_tiles;
    const int hk = id % a.kv_heads, b = id / a.kv_heads;
    const int group_of = (b * a.kv_heads + hk) * a.row_tiles + rt;  // of the workgroups that share rows
    const int row0 = rt * 16 * NQ, rows = a.rows - row0 < 16 * NQ ? a.rows - row0 : 16 * NQ;

    const int n = live_keys(a, b);
    const int64_t start = a.causal ? (a.start != nullptr ? a.start[b] : 0) : 0;
    const int64_t last = a.causal ? start + (row0 + rows - 1) / a.group : int64_t(n) - 1;
    const int64_t end64 = last + 1 < n ? last + 1 : n;
    const int end = end64 < 0 ? 0 : int(end64);
    const int64_t first64 = a.causal ? start + row0 / a.group + 1 : n;  // the first key that some row leaves out
    const int first = first64 < 0 ? 0 : first64 < n ? int(first64) : n;
    // the splits share the keys there are, not the keys there could be
    const int tiles = (end + kShortKeys - 1) / kShortKeys;
    const int t0 = int(int64_t(tiles) * split / a.splits), t1 = int(int64_t(tiles) * (split + 1) / a.splits);

    Rows<D, NQ> w;
    rows_init(w);
    load_q(w, a, b, hk, row0);
    int64_t mine[NQ];
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
        const int row = row0 + 16 * qb + l16;
        mine[qb] = a.causal ? start + (row < a.rows ? row : a.rows - 1) / a.group : int64_t(1) << 40;
    }
    const Offsets<D> f = offsets<D>();

    const uint32_t k_row = uint32_t(a.k_token) * 2u, v_row = uint32_t(a.v_token) * 2u;
    const unsigned char* kp = reinterpret_cast<const unsigned char*>(a.k + int64_t(b) * a.k_batch + int64_t(hk) * a.k_head);
    const unsigned char* vp = reinterpret_cast<const unsigned char*>(a.v + int64_t(b) * a.v_batch + int64_t(hk) * a.v_head);
    const uint8_t* mask = a.mask == nullptr ? nullptr : a.mask + int64_t(b) * a.mask_batch;
    // copy i of a wave brings rows i * kRowsPerCopy ..; their swizzles repeat every 16 rows
    const int r0 = lane / (D / 8), p0 = lane % (D / 8);
    const auto mask_rs = make_rsrc(mask, mask != nullptr ? uint32_t(n) : 0u);
    unsigned char* const at = tiles_lds[wave];
    for (int t = t0 + wave; t < t1; t += kWaves) {
        const int key0 = kShortKeys * t;
        const int have = n - key0 < kShortKeys ? n - key0 : kShortKeys;  // rows past the last key come as zeros
        const uint8_t byte = uint8_t(__builtin_amdgcn_raw_buffer_load_b8(mask_rs, uint32_t(key0 + lane), 0, 0));
        const auto kr = make_rsrc(kp + int64_t(key0) * k_row, uint32_t(have - 1) * k_row + 2u * D);
        const auto vr = make_rsrc(vp + int64_t(key0) * v_row, uint32_t(have - 1) * v_row + 2u * D);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int r = i * kRowsPerCopy + r0;
            dma16(kr, at + i * 1024, uint32_t(r) * k_row + uint32_t(p0 ^ k_swz<D>(r)) * 16u, 0);
        }
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int r = i * kRowsPerCopy + r0;
            dma16(vr, at + kTile + i * 1024, uint32_t(r) * v_row + uint32_t(p0 ^ v_swz<D>(r)) * 16u, 0);
        }
        uint64_t live = have == kShortKeys ? 0xFFFFFFFFull : (1ull << have) - 1;
        if (mask != nullptr) live = __ballot(lane < kShortKeys && byte != 0);
        Scores<2, NQ> x;
        Probs<2, NQ> p;
        uint64_t allowed[NQ];
        bool odd = false;
        const bool partial = live != 0xFFFFFFFFull || key0 + kShortKeys > first;
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");
        if (live != 0) {
            if (partial) {
#pragma unroll
                for (int qb = 0; qb < NQ; ++qb) allowed[qb] = live & up_to(mine[qb] - key0);
                odd = __any(tidy_v<D, false>(at + kTile, 0, kShortKeys, live));
            }
            scores(w, f, at, x);
            if (partial) mask_scores(x, allowed);
            probabilities_checked(w, x, p, a.scale_log2);
            if (odd) {
                add_nonfinite<D, NQ>(w, at + kTile, kShortKeys, allowed);
                tidy_v<D, true>(at + kTile, 0, kShortKeys, live);
            }
            weighted(w, f, at + kTile, p);
        }
        // the tile's reads are done before the next copies may land
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        asm volatile("" ::: "memory");
    }

    // ---- the waves' results ----
    // wave w's O in place of its tile (16 bytes per lane, column block and row block)
    f32x4_t* const mine_o = reinterpret_cast<f32x4_t*>(at);
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int qb = 0; qb < NQ; ++qb) mine_o[(d * NQ + qb) * 64 + lane] = w.o[d][qb];
    if (q == 0) {
#pragma unroll
        for (int qb = 0; qb < NQ; ++qb) {
            join_mc[wave][qb][l16] = w.mc[qb];
            join_l[wave][qb][l16] = w.l[qb][0];
        }
    }
    __syncthreads();
    const int64_t part_base = int64_t(group_of) * a.splits * (16 * NQ);
    const uint32_t part_bytes = uint32_t(a.splits) * uint32_t(rows) * (D + 2) * 4u;  // of these rows
    constexpr int kSc1 = 16;  // through to the device-coherent level: other workgroups' caches are elsewhere
    const auto part_rs = make_rsrc(a.part + part_base * (D + 2), a.splits > 1 ? part_bytes : 0u);
    auto row_factors = [&](const float* mc, const float* l, int count, int stride, float* factor, float& total) {
        float top = kNegInf;
        for (int i = 0; i < count; ++i) top = fmaxf(top, mc[i * stride]);
        total = 0.f;
        for (int i = 0; i < count; ++i) {
            factor[i] = mc[i * stride] == kNegInf ? 0.f : __builtin_amdgcn_exp2f(mc[i * stride] - top);
            total += factor[i] * l[i * stride];
        }
        return top;
    };
    // O of a row of the tile, columns col .. col + 3, divided by the sum l (0: a row without keys)
    auto store4 = [&](int in_tile, int col, f32x4_t v, float l) {
        const int row = row0 + in_tile;
        const int tok = row / a.group, g = row - tok * a.group;
        uint16_t* dst = a.o + int64_t(b) * a.o_batch + int64_t(tok) * a.o_token + int64_t(hk * a.group + g) * a.o_head + col;
        const float r = l == 0.f ? 0.f : 1.f / l;
        *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{pack_bf16(v[0] * r, v[1] * r), pack_bf16(v[2] * r, v[3] * r)};
    };
#pragma unroll
    for (int qb = 0; qb < NQ; ++qb) {
        const int row = 16 * qb + l16;
        float factor[kWaves], total;
        const float top = row_factors(&join_mc[0][qb][l16], &join_l[0][qb][l16], kWaves, NQ * 16, factor, total);
#pragma unroll
        for (int d0 = 0; d0 < D / 16; d0 += kWaves) {
            const int d = d0 + wave;
            f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                const f32x4_t u = reinterpret_cast<const f32x4_t*>(tiles_lds[i])[(d * NQ + qb) * 64 + lane];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(factor[i], u[e], v[e]);
            }
            if (row < rows) {
                if (a.splits == 1)
                    store4(row, 16 * d + 4 * q, v, total);
                else
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), part_rs,
                                                           (uint32_t(split * rows + row) * (D + 2) + uint32_t(16 * d + 4 * q)) * 4u, 0, kSc1);
            }
        }
        if (a.splits > 1 && wave == 0 && q == 0 && row < rows) {
            const uint32_t at = (uint32_t(split * rows + row) * (D + 2) + D) * 4u;
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(top), part_rs, at, 0, kSc1);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(total), part_rs, at + 4u, 0, kSc1);
        }
    }
    if (a.splits == 1) return;

    // ---- the splits' results: the last workgroup of the head to arrive joins them ----
    wait_vmcnt<0>();  // the partial result is there before the arrival counts
    __syncthreads();
    if (threadIdx.x == 0)
        last_split = __hip_atomic_fetch_add(&a.counters[group_of], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == uint32_t(a.splits - 1);
    __syncthreads();
    if (!last_split) return;
    if (threadIdx.x == 0) __hip_atomic_store(&a.counters[group_of], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // (row, 4 columns) per thread, with the splits in `parts` ranges where threads are left over; kAhead loads in
    // flight, the first of them while the rows' factors are worked out
    constexpr int kAhead = 16;
    const int items = rows * (D / 4);
    int parts = 1;
    while (parts < 4 && 2 * parts * items <= 64 * kWaves) parts *= 2;
    const int span = (a.splits + parts - 1) / parts;
    f32x4_t u[kAhead];
    auto fetch = [&](int i, int s0, int s1) __attribute__((always_inline)) {
        const int item = i % items;
        const uint32_t at = (uint32_t(item / (D / 4)) * (D + 2) + 4u * uint32_t(item % (D / 4))) * 4u;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)  // a split past the range reads as zeros
            u[j] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                   part_rs, s0 + j < s1 ? uint32_t((s0 + j) * rows) * (D + 2) * 4u + at : 0xFFFFFF00u, 0, kSc1));
    };
    auto range_end = [&](int part) { return (part + 1) * span < a.splits ? (part + 1) * span : a.splits; };
    const int mine_i = int(threadIdx.x);
    if (mine_i < items * parts) fetch(mine_i, mine_i / items * span, range_end(mine_i / items));
    float* const factors = reinterpret_cast<float*>(tiles_lds);  // [rows][splits], then the sums [rows]
    float* const totals = factors + rows * a.splits;
    for (int row = wave; row < rows; row += kWaves) {  // a lane per split (kMaxShortSplits at most)
        const uint32_t at = (uint32_t(lane * rows + row) * (D + 2) + D) * 4u;
        const bool in = lane < a.splits;
        const float mc = in ? __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(part_rs, at, 0, kSc1)) : kNegInf;
        const float l = in ? __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(part_rs, at + 4u, 0, kSc1)) : 0.f;
        float top = mc;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
        const float fac = mc == kNegInf ? 0.f : __builtin_amdgcn_exp2f(mc - top);
        float sum = fac * l;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
        if (in) factors[row * a.splits + lane] = fac;
        if (lane == 0) totals[row] = sum;
    }
    __syncthreads();
    f32x4_t* const sums = reinterpret_cast<f32x4_t*>(tiles_lds[2]);  // [parts][items]
    for (int i = mine_i; i < items * parts; i += 64 * kWaves) {
        const int part = i / items, item = i - part * items;
        const int row = item / (D / 4), col = 4 * (item % (D / 4));
        const int s1 = range_end(part);
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        for (int s0 = part * span; s0 < s1; s0 += kAhead) {
            if (i != mine_i || s0 != part * span) fetch(i, s0, s1);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float fac = s0 + j < s1 ? factors[row * a.splits + s0 + j] : 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(fac, u[j][e], v[e]);
            }
        }
        if (parts == 1)
            store4(row, col, v, totals[row]);
        else
            sums[i] = v;
    }
    if (parts == 1) return;
    __syncthreads();
    for (int item = int(threadIdx.x); item < items; item += 64 * kWaves) {
        f32x4_t v = sums[item];
        for (int part = 1; part < parts; ++part) {
            const f32x4_t u = sums[part * items + item];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += u[e];
        }
        store4(item / (D / 4), 4 * (item % (D / 4)), v, totals[item / (D / 4)]);
    }
}

// Joins the splits' partial results of a row, in split order: a wave per row.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a) {
    const int lane = int(threadIdx.x) & 63;
    const int64_t id = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (id >= int64_t(a.batch) * a.kv_heads * a.rows) return;
    const int row = int(id % a.rows);
    const int64_t bh = id / a.rows;
    const int64_t base = bh * a.splits * a.rows + row;
    float m = kNegInf;
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_ml[2 * (base + int64_t(s) * a.rows)]);
    float l = 0.f, o[D / 64];
#pragma unroll
    for (int e = 0; e < D / 64; ++e) o[e] = 0.f;
    for (int s = 0; s < a.splits; ++s) {
        const int64_t r = base + int64_t(s) * a.rows;
        const float ms = a.part_ml[2 * r];
        const float f = ms == kNegInf ? 0.f : __builtin_amdgcn_exp2f(ms - m);
        l += f * a.part_ml[2 * r + 1];
#pragma unroll
        for (int e = 0; e < D / 64; ++e) o[e] = __builtin_fmaf(f, a.part[r * D + (D / 64) * lane + e], o[e]);
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    const int b = int(bh / a.kv_heads), hk = int(bh % a.kv_heads);
    const int t = row / a.group, g = row - t * a.group;
    uint16_t* dst = a.o + int64_t(b) * a.o_batch + int64_t(t) * a.o_token + int64_t(hk * a.group + g) * a.o_head;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) dst[(D / 64) * lane + e] = float_to_bf16_bits(o[e] * f);
}

// The launch log's line of an attention kernel.
void trace_attention(const char* form, int tile_rows, const AttnArgs& a, int head_dim, unsigned grid) {
    std::fprintf(stderr, "lowbit: attention %s rows=%d splits=%d grid=%u block=256 problem=%dx%dx%dx%d kv_heads=%d dim=%d%s\n", form,
                 tile_rows, a.splits, grid, a.batch, a.rows / a.group, a.kv_len, a.kv_heads * a.group, a.kv_heads, head_dim,
                 a.causal ? " causal" : "");
}

template <int D>
hipError_t launch_d(const AttnArgs& a, const AttnPlan& plan, hipStream_t stream) {
    if (plan.is_short) {
        const unsigned grid = unsigned(a.row_tiles) * unsigned(a.splits) * unsigned(a.kv_heads) * unsigned(a.batch);
        if (a.rows <= 16)
            hipLaunchKernelGGL((attention_short_kernel<D, 1>), dim3(grid), dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((attention_short_kernel<D, 2>), dim3(grid), dim3(256), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e == hipSuccess && trace_enabled()) trace_attention("few", a.rows <= 16 ? 16 : 32, a, D, grid);
        return e;
    }
    const int64_t grid = int64_t(a.row_tiles) * a.splits * a.kv_heads * a.batch;
    if (plan.tile_rows == 64)
        hipLaunchKernelGGL((attention_kernel<D, 1>), dim3(unsigned(grid)), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((attention_kernel<D, 2>), dim3(unsigned(grid)), dim3(256), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && trace_enabled()) trace_attention("many", plan.tile_rows, a, D, unsigned(grid));
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t rows = int64_t(a.batch) * a.kv_heads * a.rows;
    hipLaunchKernelGGL((attention_join_kernel<D>), dim3(unsigned((rows + 3) / 4)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

constexpr int kMaxShortSplits = 64;     // a lane per split in the join

}  // namespace

// Which kernel, and how the keys are split: the one whose estimated time is less (one row block, 16 or 32 rows,
// always goes to the few-rows kernel).  The estimates (us, D = 64 / 128) are fits to measured calls of 8 to 96 heads, 64 to
// 4608 rows and 200 to 8192 keys: in five of 108 of them the other kernel is 9% to 13% faster, in the rest less or
// not (profiles/attention_plan_estimates.txt).  They plan with kv_len: with key_lens far below it the few-rows kernel may
// be the faster one, and 1000 causal queries at the end of 2000 to 8000 keys, 16 heads, without a workspace, are 10% to 20%
// slower than there.  Measured (few / many, us): 256 x 1024, 24 heads of 128: 15 / 18; 512 x 2048, 16 heads of 128: 26 / 30; 512 x 512, 24
// heads of 128: 14 / 12; 1024 x 1024, 24 heads of 128: 32 / 25, of 64: 17 / 16; 4 x 512 x 512, 24 heads of 128: 37 / 25.
//   LOWBIT_ATTENTION=few|many|many64|many128 in the environment forces the kernel, or also its rows (A/B runs and tests).
//
// The few-rows kernel (32 rows per workgroup, its waves over the keys, two or three workgroups per compute unit):
// 6.2 / 7, 0.0049 / 0.0093 a key for a workgroup alone on its compute unit, 0.45 of that for each beside it, and 4.5 / 6
// for each further round.  Keys are split until every compute unit has a workgroup of three tiles a wave at least
// (512 workgroups were slower at 1024 rows, 27 against 17, and at 40007 keys, 33 against 32); the join costs 10 / 12.
double few_us(int64_t groups, int64_t keys, bool joins, int head_dim) {
    const int64_t room = kComputeUnits * (head_dim == 64 ? 3 : 2);
    auto load = [](int64_t n) { return n <= kComputeUnits ? 1.0 : 0.55 + 0.45 * double(n) / kComputeUnits; };
    const int64_t rounds = groups == 0 ? 0 : (groups - 1) / room;  // full ones before the last
    return (head_dim == 64 ? 6.2 : 7.0) + (joins ? head_dim == 64 ? 10.0 : 12.0 : 0.0) + double(rounds) * (head_dim == 64 ? 4.5 : 6.0) +
           double(keys) * (head_dim == 64 ? 0.0049 : 0.0093) * (double(rounds) * load(room) + load(groups - rounds * room));
}
// The other kernel: a start, and a time per tile of 64 keys for a compute unit that has up to n = ceil(groups / 256)
// workgroups: 5 / 9 and 0.79 / 1.16 of one of 128 rows alone, times 0.75 n from two on.  With 64 rows at a time 5 / 5.5,
// and as in the table: they fill the units more evenly, and four of them of D = 64 fit one; but they read twice as
// much LDS per product.  Measured (128 / 64 rows, us): 2 x 1533 x 1533, 16 heads of 64: 33 / 30; 4 x 300 x 300, 24
// heads of 128: 21 / 14; 4608 x 4608, 24 heads of 128: 267 / 313; causal 1533 x 1533, 24 heads of 128: 44 / 31, 4608 x
// 4608: 163 / 174.
double many_us(int64_t tiles, int64_t groups, int tile_rows, int head_dim) {
    const double n = double(tiles_of(groups, kComputeUnits)), whole = head_dim == 64 ? 0.79 : 1.16;
    if (tile_rows == 128) return (head_dim == 64 ? 5.0 : 9.0) + double(tiles) * whole * (n <= 1 ? 1.0 : 0.75 * n);
    if (head_dim == 64) return 5.0 + double(tiles) * whole * (0.1 + 0.42 * n);
    return 5.5 + double(tiles) * whole * (n <= 1 ? 0.7 : n <= 2 ? 1.0 : 0.3 + 0.48 * n);
}
// Keys split: two workgroups of 128 rows per compute unit, of four tiles at least; the join costs 8 / 7, 0.4 / 0.15 a
// split, and 7 / 14 for 512 workgroups' parts to go to memory and back.
double join_us(int64_t groups, int64_t splits, int head_dim) {
    return (head_dim == 64 ? 8.0 : 7.0) + (head_dim == 64 ? 0.4 : 0.15) * double(splits) + (head_dim == 64 ? 7.0 : 14.0) * double(groups) / (2 * kComputeUnits);
}

// may_split false: no workspace to split with.  Of a's arrays only whether they are there counts.
AttnPlan plan_attention(const AttnArgs& a, int head_dim, bool may_split) {
    const int64_t batch = a.batch, kv_heads = a.kv_heads, rows = a.rows, kv_len = a.kv_len;
    // few rows
    const int64_t few_rows = rows <= 16 ? 16 : 32, few_groups = batch * kv_heads * tiles_of(rows, few_rows);
    const int64_t few_tiles = tiles_of(kv_len, kShortKeys);
    int64_t few_splits = few_groups >= kComputeUnits || few_groups == 0 ? 1 : kComputeUnits / few_groups;
    few_splits = few_splits < few_tiles / 12 ? few_splits : few_tiles / 12;
    few_splits = few_splits < kMaxShortSplits ? few_splits : kMaxShortSplits;
    few_splits = few_splits < 1 || !may_split ? 1 : few_splits;
    const double few = few_us(few_groups * few_splits, tiles_of(few_tiles, few_splits) * kShortKeys, few_splits > 1, head_dim);
    // many rows
    const int64_t groups = batch * kv_heads * tiles_of(rows, 128), halves = batch * kv_heads * tiles_of(rows, 64);
    const int64_t tiles = tiles_of(kv_len, 64);
    const double full = many_us(tiles, groups, 128, head_dim), half = many_us(tiles, halves, 64, head_dim);
    int tile_rows = halves <= kMaxGrid256 && half < full ? 64 : 128;
    double many = tile_rows == 64 ? half : full;
    int64_t splits = groups >= kComputeUnits || groups == 0 || !may_split ? 1 : 2 * kComputeUnits / groups;
    splits = splits < tiles / 4 ? splits : tiles / 4;
    if (splits > 1) {
        const double joined = many_us(tiles_of(tiles, splits), groups * splits, 128, head_dim) + join_us(groups * splits, splits, head_dim);
        if (joined < many) {
            many = joined;
            tile_rows = 128;
        } else {
            splits = 1;
        }
    }
    splits = splits < 1 ? 1 : splits;
    // Causal, all row tiles resident at once: those with the most keys decide, and 64 rows share the keys out more evenly,
    // while the keys are few beside the queries.  In a chunk of queries after a long cache every tile has about as many
    // keys, and the estimates above hold.  Measured, queries at the end of 1, 1.5, 2, 3, 4 and 8 times as many keys (64 / 128
    // rows, us): 2560 queries, 24 heads of 128 69 / 77, 109 / 113, 155 / 148, 248 / 218, 337 / 288, 710 / 580; 4096, 16 of 128 92 / 121, 171 / 178,
    // 248 / 237, 401 / 355, 544 / 470, 1177 / 948; 2560, 24 of 64 40 / 47, 63 / 69, 86 / 90, 134 / 134, 184 / 176, 380 / 348.  (The
    // workspace's size and the kernel do not depend on it.)
    const int64_t queries = rows / a.group, reach = a.start == nullptr && queries < kv_len ? queries : kv_len;
    if (a.causal && splits == 1 && groups <= 2 * kComputeUnits && halves <= kMaxGrid256 &&
        4 * reach <= (head_dim == 64 ? 12 : 7) * queries)
        tile_rows = 64;

    AttnPlan p{};
    p.is_short = rows <= 32 || (few <= many && few_groups <= kMaxGrid256);
    if (const char* force = std::getenv("LOWBIT_ATTENTION")) {
        if (std::strcmp(force, "few") == 0) p.is_short = true;
        if (std::strncmp(force, "many", 4) == 0) p.is_short = false;
        if (std::strcmp(force, "many128") == 0) tile_rows = 128;
        if (std::strcmp(force, "many64") == 0 && halves <= kMaxGrid256) {
            tile_rows = 64;
            splits = 1;
        }
    }
    if (p.is_short) {
        p.row_tiles = int(tiles_of(rows, few_rows));
        p.splits = int(few_splits);
    } else {
        p.tile_rows = tile_rows;
        p.row_tiles = int(tiles_of(rows, tile_rows));
        const int64_t share = tiles_of(tiles, splits);  // no more splits than have a tile
        p.splits = share > 0 ? int(tiles_of(tiles, share)) : 1;
    }
    const int64_t padded = p.is_short ? int64_t(p.row_tiles) * (rows <= 16 ? 16 : 32) : rows;
    p.part_rows = p.splits > 1 ? batch * kv_heads * padded * p.splits : 0;
    p.bytes = p.splits > 1 ? kWorkspaceCounterBytes + size_t(p.part_rows) * (size_t(head_dim) + 2) * 4u : 0;
    return p;
}

hipError_t launch_attention(AttnArgs a, int head_dim, const AttnPlan& plan, void* workspace, hipStream_t stream) {
    a.row_tiles = plan.row_tiles;
    a.splits = plan.splits;
    a.counters = static_cast<uint32_t*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kWorkspaceCounterBytes);
    a.part_ml = a.part + plan.part_rows * head_dim;
    return head_dim == 64 ? launch_d<64>(a, plan, stream) : launch_d<128>(a, plan, stream);
}

}  // namespace lowbit
