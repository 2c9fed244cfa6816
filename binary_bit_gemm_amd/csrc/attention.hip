// Attention over grouped heads: O = softmax(scale * Q K^T, over the allowed keys) V.
//
// Row r of a kv head's problem is query token r / G of its q head r % G (G q heads share a kv head), so
// the heads of a group read each key and value once, also where there is one query token.  Keys go by
// in tiles, with the running maximum m and sum l of the softmax per row (one pass):
//     p = exp2(c s - c m),  l += sum p,  O += p v,      c = scale * log2(e);
// where m grows, l and O are multiplied by exp2(c m_old - c m_new).
//
// The products are computed transposed, S^T = K Q^T and O^T = V^T P^T, with 32x32x16 MFMAs: a lane
// then holds 16 scores of one query per 32 keys (lane l: query l % 32, keys 8 (i / 4) + 4 (l / 32) + i % 4),
// so the row maximum is an in-lane maximum and one exchange between the two lane halves, the
// factors of m and l are one number per lane, and the probabilities, rounded to bf16 in pairs, are
// already the B operand of the second product: its K order is the order in which the lane holds
// them, and V^T is read from LDS in that order by transposing reads (4 keys x 16 columns each).
//
// Rounding to bf16: the probabilities before the second product (the matrix cores' input; relative
// 2^-8 each, averaged over the keys) and O at the store.  Scores, m, l and O are fp32.
#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

constexpr float kNegInf = -__builtin_inff();
// A maximum that grows by less than this (in powers of two) leaves m as it is: p then reaches 2^8
// instead of 1, which fp32 sums and the bf16 mantissa do not notice, and O is not rescaled.
constexpr float kLazy = 8.f;

// ---- layouts in LDS: rows of D elements in 16-byte chunks, chunk c of row r at position c ^ swz(r) ----
// K is read 16 bytes per lane from 32 consecutive rows at one chunk; 16 rows must land in 16 different
// 16-byte bank groups of the 256-byte line.
template <int D>
__device__ __forceinline__ int k_swz(int r) {
    return D == 128 ? (r & 15) : ((r >> 1) & 7);
}
// V is read by transposing reads, 8 bytes per lane: 16 lanes take 4 rows x 32 bytes, the wave instruction
// rows 4h .. 4h+3 x 64 bytes.  The four rows' 64-byte windows must not share banks.
template <int D>
__device__ __forceinline__ int v_swz(int r) {
    return D == 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
}

// One wave's state for 32 rows.
template <int D>
struct Rows {
    bf16x8_t q[D / 16];   // B operand: lane (query l % 32, h): elements 16 kk + 8 h ..
    f32x16_t o[D / 32];   // O^T
    float m, l;           // the softmax's maximum (raw scores) and the lane half's share of its sum
};

template <int D>
__device__ __forceinline__ void rows_init(Rows<D>& w) {
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) w.o[b][i] = 0.f;
    w.m = kNegInf;
    w.l = 0.f;
}

__device__ __forceinline__ float other_half(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// The lane's byte offsets into a K and a V tile, without the constants that the compiler folds into the
// instructions: K row l % 32 at chunk 2 kk + h (rows 32 apart have the same swizzle), V row 4 h +
// (l % 16) / 4 at column block b (rows 4 apart as well).
template <int D>
struct Offsets {
    int k[D / 16], v[D / 32];
};

template <int D>
__device__ __forceinline__ Offsets<D> offsets() {
    const int lane = int(threadIdx.x) & 63;
    const int l32 = lane & 31, h = lane >> 5, i16 = lane & 15, dsel = (lane >> 4) & 1;
    Offsets<D> f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) f.k[kk] = l32 * (2 * D) + (((2 * kk + h) ^ k_swz<D>(l32)) << 4);
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
        const int r = 4 * h + (i16 >> 2), chunk = 4 * b + 2 * dsel + ((i16 & 3) >> 1);
        f.v[b] = r * (2 * D) + ((chunk ^ v_swz<D>(r)) << 4) + 8 * (i16 & 1);
    }
    return f;
}

// Scores of NKB * 32 keys of the K tile at kt.
template <int D, int NKB>
__device__ __forceinline__ void scores(const Rows<D>& w, const Offsets<D>& f, const unsigned char* kt, f32x16_t (&s)[NKB]) {
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                *reinterpret_cast<const bf16x8_t*>(kt + f.k[kk] + kb * 32 * (2 * D)), w.q[kk], s[kb], 0, 0, 0);
    }
}

// Scores of keys that the lane's query does not take (bit of `allowed` clear) to -inf.
template <int NKB>
__device__ __forceinline__ void mask_scores(f32x16_t (&s)[NKB], uint64_t allowed) {
    asm volatile("");  // a branch, not a select in every tile
    const uint64_t mine = allowed >> ((threadIdx.x & 32) >> 3);
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb) {
        const uint32_t bits = uint32_t(mine >> (32 * kb));
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] = (bits >> (8 * (i / 4) + i % 4)) & 1u ? s[kb][i] : kNegInf;
    }
}

// Largest score of the lane's row among s.
template <int NKB>
__device__ __forceinline__ float row_max(const f32x16_t (&s)[NKB]) {
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kb][i]);
    return fmaxf(top, other_half(top));
}

// m grows to `top` where a row of the wave needs it, and l and O follow.
template <int D>
__device__ __forceinline__ void grow(Rows<D>& w, float top, float c) {
    if (__any((top - w.m) * c > kLazy || (w.m == kNegInf && top != kNegInf))) {
        const float m = fmaxf(w.m, top);
        const float f = m == kNegInf ? 1.f : __builtin_amdgcn_exp2f((w.m - m) * c);
        w.m = m;
        w.l *= f;
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) w.o[b][i] *= f;
    }
}

// What the exponents subtract: c m, and 0 for a row that has no key yet (its scores are -inf).
template <int D>
__device__ __forceinline__ float offset(const Rows<D>& w, float c) {
    return w.m == kNegInf ? 0.f : w.m * c;
}

// s becomes the probabilities to the maximum so far, l their sum.
template <int D, int NKB>
__device__ __forceinline__ void probabilities(Rows<D>& w, f32x16_t (&s)[NKB], float c) {
    const float mc = offset(w, c);
    float sum = 0.f;
#pragma unroll
    for (int kb = 0; kb < NKB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[kb][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][i], c, -mc));
            sum += s[kb][i];
        }
    w.l += sum;
}

// O += P V for the V tile at vt.
template <int D, int NKB>
__device__ __forceinline__ void weighted(Rows<D>& w, const Offsets<D>& f, const unsigned char* vt, const f32x16_t (&s)[NKB]) {
#pragma unroll
    for (int k2 = 0; k2 < 2 * NKB; ++k2) {  // 16 keys each
        bf16x8_t p;
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = static_cast<__bf16>(s[k2 / 2][8 * (k2 % 2) + i]);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            s16x4_t v[2];
#pragma unroll
            for (int part = 0; part < 2; ++part)
                v[part] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4_t*)(vt + f.v[b] + (16 * k2 + 8 * part) * (2 * D)));
            const s16x8_t a = __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
            w.o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), p, w.o[b], 0, 0, 0);
        }
    }
}

__device__ __forceinline__ bool pair_finite(uint32_t v) { return (v & 0x7F80u) != 0x7F80u && (v & 0x7F800000u) != 0x7F800000u; }

// One tile's probabilities and values and the next tile's scores in one block of code, so that the matrix cores
// have work while the vector unit takes the exponentials: s (scores of the tile whose values are at
// vt) is used up, sn becomes the scores of the K tile at kt; the result is the rows' largest new score.
template <int D>
__device__ __forceinline__ float fused_step(Rows<D>& w, const Offsets<D>& f, const unsigned char* kt, const unsigned char* vt,
                                            f32x16_t (&s)[2], f32x16_t (&sn)[2], float c) {
    scores<D, 2>(w, f, kt, sn);
    probabilities<D, 2>(w, s, c);
    weighted<D, 2>(w, f, vt, s);
    return row_max<2>(sn);
}

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
template <int D>
__device__ __forceinline__ void add_nonfinite(Rows<D>& w, const unsigned char* vt, int keys, uint64_t allowed) {
    int h = (int(threadIdx.x) >> 5) & 1;
    asm volatile("" : "+v"(h));
    for (int j = 0; j < keys; ++j) {
        const bool mine = (allowed >> j) & 1;
        if (!__any(mine)) continue;
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const u32x2_t v = *reinterpret_cast<const u32x2_t*>(vt + j * (2 * D) + (((4 * b + e) ^ v_swz<D>(j)) << 4) + 8 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t bits = i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16;
                    if (mine && (bits & 0x7F800000u) == 0x7F800000u) w.o[b][4 * e + i] += __uint_as_float(bits);
                }
            }
    }
}

// The rows' Q operands (rows past the last read as zeros).
template <int D>
__device__ __forceinline__ void load_q(Rows<D>& w, const AttnArgs& a, int b, int hk, int row) {
    const int h = (int(threadIdx.x) >> 5) & 1;
    const bool in = row < a.rows;
    const int t = in ? row / a.group : 0, g = in ? row - t * a.group : 0;
    const uint16_t* src = a.q + int64_t(b) * a.q_batch + int64_t(t) * a.q_token + int64_t(hk * a.group + g) * a.q_head;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        u32x4_t v = {0, 0, 0, 0};
        if (in) v = *reinterpret_cast<const u32x4_t*>(src + 16 * kk + 8 * h);
        w.q[kk] = __builtin_bit_cast(bf16x8_t, v);
    }
}

// O of one row (its lane pair) to memory, scaled by f: 16 bytes per lane and 32 columns after an exchange
// between the lane halves (each half holds 4 of every 8 consecutive columns).
template <int D>
__device__ __forceinline__ void store_o(const Rows<D>& w, const AttnArgs& a, int b, int hk, int row, float f) {
    const int h = (int(threadIdx.x) >> 5) & 1;
    const bool in = row < a.rows;
    const int t = in ? row / a.group : 0, g = in ? row - t * a.group : 0;
    uint16_t* dst = a.o + int64_t(b) * a.o_batch + int64_t(t) * a.o_token + int64_t(hk * a.group + g) * a.o_head;
    auto pair = [&](float x, float y) {
        return uint32_t(float_to_bf16_bits(x * f)) | (uint32_t(float_to_bf16_bits(y * f)) << 16);
    };
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // columns 32 d + 16 e + (0..7 | 8..15), four of each eight per half
            const uint32_t x0 = pair(w.o[d][8 * e], w.o[d][8 * e + 1]), x1 = pair(w.o[d][8 * e + 2], w.o[d][8 * e + 3]);
            const uint32_t y0 = pair(w.o[d][8 * e + 4], w.o[d][8 * e + 5]), y1 = pair(w.o[d][8 * e + 6], w.o[d][8 * e + 7]);
            const auto s0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
            if (in) *reinterpret_cast<u32x4_t*>(dst + 32 * d + 16 * e + 8 * h) = u32x4_t{s0[0], s1[0], s0[1], s1[1]};
        }
}

// Partial results of one row for the join: O unnormalised, then (c m, l).
template <int D>
__device__ __forceinline__ void store_part(const Rows<D>& w, const AttnArgs& a, int64_t part_row, bool in, float l) {
    const int h = (int(threadIdx.x) >> 5) & 1;
    if (!in) return;
    float* dst = a.part + part_row * D;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<f32x4_t*>(dst + 32 * d + 8 * e + 4 * h) =
                f32x4_t{w.o[d][4 * e], w.o[d][4 * e + 1], w.o[d][4 * e + 2], w.o[d][4 * e + 3]};
    if (h == 0) {
        a.part_ml[2 * part_row] = w.m == kNegInf ? kNegInf : w.m * a.scale_log2;
        a.part_ml[2 * part_row + 1] = l;
    }
}

// Keeps a wave-uniform value in a scalar register: without it the compiler reloads kernel arguments inside
// the loop, and a scalar load shares its wait with every LDS read in flight.
template <class T>
__device__ __forceinline__ T in_sgpr(T v) {
    asm volatile("" : "+s"(v));
    return v;
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

// Long rows: a workgroup of 4 waves takes 128 rows of one kv head, a wave 32 of them; tiles of 64 keys go
// through LDS, double-buffered, by direct copies one tile ahead.
template <int D>
__global__ __launch_bounds__(256, 2) void attention_kernel(AttnArgs a) {
    constexpr int kTile = 64 * D * 2;
    constexpr int kRowsPerCopy = 512 / D;         // rows that one wave-wide 16-byte copy brings
    constexpr int kCopies = 64 / kRowsPerCopy / 4;  // copies per wave and tile
    // an array per buffer, not one indexed by parity: the compiler then sees that a tile's reads do not
    // depend on the copies still landing in the other buffer
    __shared__ __attribute__((aligned(1024))) unsigned char kbuf0[kTile], kbuf1[kTile], vbuf0[kTile], vbuf1[kTile];
    __shared__ int odd_tile;  // the last tile in which an infinity or a NaN was seen
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    // tiles of one head next to each other, heads of one XCD together
    int id = xcd_remap(int(blockIdx.x), int(gridDim.x));
    const int rt = id % a.row_tiles;
    id /= a.row_tiles;
    const int split = id % a.splits;
    id /= a.splits;
    const int hk = id % a.kv_heads, b = id / a.kv_heads;

    const int n = in_sgpr(live_keys(a, b));
    const int row = rt * 128 + wave * 32 + (lane & 31);
    const int64_t start = a.causal ? (a.start != nullptr ? a.start[b] : 0) : 0;
    // the last key of the workgroup's and of the lane's rows
    const int last_row = rt * 128 + 127 < a.rows ? rt * 128 + 127 : a.rows - 1;
    const int64_t last = a.causal ? start + last_row / a.group : int64_t(n) - 1;
    const int64_t mine = a.causal ? start + (row < a.rows ? row : a.rows - 1) / a.group : int64_t(1) << 40;
    // the first key that a row of the workgroup leaves out by the causal rule (all rows take those before)
    const int64_t first64 = a.causal ? start + (rt * 128) / a.group + 1 : n;
    const int64_t end64 = last + 1 < n ? last + 1 : n;
    const int end = end64 < 0 ? 0 : int(end64);
    const int first = in_sgpr(first64 < 0 ? 0 : first64 < n ? int(first64) : n);
    const int tiles = (end + 63) / 64;
    const int t0 = split * a.tiles_per_split;
    const int t1 = in_sgpr(t0 + a.tiles_per_split < tiles ? t0 + a.tiles_per_split : tiles);

    Rows<D> w;
    rows_init(w);
    load_q(w, a, b, hk, row);
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
    // The lane's bytes of the mask for tiles t, t + 1 and t + 2, fetched before they are needed.
    auto fetch = [&](int t) __attribute__((always_inline)) {
        return mask != nullptr && 64 * t + lane < n ? mask[64 * t + lane] : uint8_t(0);
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
        uint64_t allowed = ~0ull;
        bool odd = false;
        if (partial) {
            allowed = live & up_to(mine - 64 * int64_t(t - 1));
            if (tidy_v<D, false>(vc, wave * 16, 16, live)) odd_tile = t;
            lds_writes_barrier();
            odd = odd_tile == t;
        }
        f32x16_t s[2];
        scores<D, 2>(w, f, kc, s);
        if (partial) mask_scores<2>(s, allowed);
        grow(w, row_max<2>(s), c);
        probabilities<D, 2>(w, s, c);
        if (odd) {
            add_nonfinite<D>(w, vc, 64, allowed);
            lds_writes_barrier();
            tidy_v<D, true>(vc, wave * 16, 16, live);
            lds_writes_barrier();
        }
        weighted<D, 2>(w, f, vc, s);
    };

    issue_k(t0, kbuf0);
    issue_v(t0, vbuf0);
    while (t < t1) {
        if (whole(t, m0) && whole(t + 1, m1) && whole(t + 2, m2)) {
            // a run of whole tiles, two per turn; the scores are one tile ahead of the values
            arrive();
            issue_k(t + 1, kbuf1);
            f32x16_t s0[2], s1[2];
            scores<D, 2>(w, f, kbuf0, s0);
            grow(w, row_max<2>(s0), c);
            do {
                arrive();
                issue_k(t + 2, kbuf0);
                issue_v(t + 1, vbuf1);
                grow(w, fused_step<D>(w, f, kbuf1, vbuf0, s0, s1, c), c);
                arrive();
                issue_k(t + 3, kbuf1);
                issue_v(t + 2, vbuf0);
                m0 = m2;
                m1 = fetch(t + 3);
                m2 = fetch(t + 4);
                grow(w, fused_step<D>(w, f, kbuf0, vbuf1, s1, s0, c), c);
                t += 2;
            } while (whole(t + 1, m1) && whole(t + 2, m2));
            arrive();
            issue_v(t + 1, vbuf1);
            probabilities<D, 2>(w, s0, c);
            weighted<D, 2>(w, f, vbuf0, s0);
            m0 = m1;
            m1 = m2;
            m2 = fetch(t + 3);
            ++t;
        } else {
            any_step(kbuf0, vbuf0, kbuf1, vbuf1);
        }
        if (t < t1) any_step(kbuf1, vbuf1, kbuf0, vbuf0);
    }
    const float l = w.l + other_half(w.l);
    if (a.splits == 1) {
        store_o(w, a, b, hk, row, l > 0.f || l != l ? 1.f / l : 0.f);
    } else {
        const int64_t base = ((int64_t(b) * a.kv_heads + hk) * a.splits + split) * a.rows;
        store_part(w, a, base + row, row < a.rows, l);
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
    const float f = l > 0.f || l != l ? 1.f / l : 0.f;
    const int b = int(bh / a.kv_heads), hk = int(bh % a.kv_heads);
    const int t = row / a.group, g = row - t * a.group;
    uint16_t* dst = a.o + int64_t(b) * a.o_batch + int64_t(t) * a.o_token + int64_t(hk * a.group + g) * a.o_head;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) dst[(D / 64) * lane + e] = float_to_bf16_bits(o[e] * f);
}

template <int D>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
    const int64_t grid = int64_t(a.row_tiles) * a.splits * a.kv_heads * a.batch;
    hipLaunchKernelGGL((attention_kernel<D>), dim3(unsigned(grid)), dim3(256), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t rows = int64_t(a.batch) * a.kv_heads * a.rows;
    hipLaunchKernelGGL((attention_join_kernel<D>), dim3(unsigned((rows + 3) / 4)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

// Splits along the keys: where the row tiles leave compute units idle, about two workgroups per
// compute unit, each with four key tiles at least.
AttnPlan plan_attention(int64_t batch, int64_t kv_heads, int64_t rows, int64_t kv_len, int head_dim) {
    AttnPlan p;
    p.row_tiles = int(tiles_of(rows, 128));
    const int64_t tiles = tiles_of(kv_len, 64), base = batch * kv_heads * p.row_tiles;
    int64_t splits = base >= kComputeUnits ? 1 : 2 * kComputeUnits / base;
    const int64_t most = tiles / 4;
    splits = splits < most ? splits : most;
    splits = splits < 1 ? 1 : splits;
    p.tiles_per_split = int(tiles_of(tiles, splits));
    p.splits = int(tiles_of(tiles, p.tiles_per_split > 0 ? p.tiles_per_split : 1));
    if (p.splits < 1) p.splits = 1;
    p.part_rows = p.splits > 1 ? batch * kv_heads * rows * p.splits : 0;
    p.bytes = size_t(p.part_rows) * (size_t(head_dim) + 2) * 4u;
    return p;
}

AttnPlan plan_attention_unsplit(AttnPlan p, int64_t kv_len) {
    p.splits = 1;
    p.tiles_per_split = int(tiles_of(kv_len, 64));
    p.part_rows = 0;
    p.bytes = 0;
    return p;
}

hipError_t launch_attention(AttnArgs a, int head_dim, const AttnPlan& plan, void* workspace, hipStream_t stream) {
    a.row_tiles = plan.row_tiles;
    a.splits = plan.splits;
    a.tiles_per_split = plan.tiles_per_split;
    a.part = static_cast<float*>(workspace);
    a.part_ml = a.part + plan.part_rows * head_dim;
    return head_dim == 64 ? launch_d<64>(a, stream) : launch_d<128>(a, stream);
}

}  // namespace lowbit
