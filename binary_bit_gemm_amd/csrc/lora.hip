// First product of the low-rank adapters beside a packed GEMM: U[m] = alpha_e * A_e X[m] for the adapter e of
// row m, with X [M, K] bf16, A [adapters, rank, K] bf16 and alpha fp32.  The second product (U B_e^T) is where the packed GEMM's
// sums start (lora_device.h).
//
// A workgroup takes 16 rows, `stack` of the adapters among them (in ascending order, blockIdx.y counting the groups; one
// past the last leaves at once), whose rank rows it stacks, and a range of K; rows of many requests cost
// more workgroups, not a longer one.  Its waves take steps of 128 of K in turn.  A step's pieces of the 16 rows of X and the rank
// rows of A, 256 bytes a row, are copied into the wave's part of LDS (four whole rows per instruction: loads straight into
// operand registers would touch 16 rows each, and took 26 us where this takes 10: 509 rows, K = 9216,
// rank 32) and multiplied in 16x16x32 blocks.  The waves' fp32 sums are added in wave order; where K is
// split across workgroups (few rows, long K) each leaves its sums in the workspace and the last to arrive adds
// them in order.  U is stored as hi + lo bf16 pairs.
#include "lora_device.h"
#include "lowbit_device.h"
#include "lowbit_internal.h"

namespace lowbit {
namespace {

constexpr int kStepK = 128;             // of K per wave and step
constexpr int kBlock = 16 * kStepK * 2;  // bytes of 16 rows' pieces: 4 KB
constexpr int kMaxStack = 2;            // adapters of a workgroup

// Chunk c (16 bytes) of row r of a 16-row block sits at position c ^ r: the 16 rows that an operand read
// touches at one chunk (k_chunk) then lie in 16 different bank groups.

// RB: blocks of 16 of the rank (the last may be half used).
template <int RB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void lora_shrink_kernel(ShrinkArgs a) {
    __shared__ __attribute__((aligned(1024))) unsigned char lds[WAVES][(1 + RB) * kBlock];
    __shared__ int last_split;
    const int lane = int(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int q = lane >> 4, l16 = lane & 15;
    const int64_t row0 = int64_t(blockIdx.x) * 16;
    const int have = a.M - row0 < 16 ? int(a.M - row0) : 16;
    int id = l16 < have ? a.rows[row0 + l16] : -1;
    id = id >= 0 && id < a.adapters ? id : -1;
    // the workgroup's adapters: those of the 16 rows from the (blockIdx.y * stack)-th on; the last repeats where there are fewer
    int cur = -1, list[kMaxStack], mine_at = -1;  // mine_at: where the lane's row finds its adapter
#pragma unroll
    for (int j = 0; j < kMaxStack; ++j) list[j] = -1;
    for (int j = 0; j < int(blockIdx.y) * a.stack; ++j) {
        cur = min_of_16(id > cur ? id : 0x7FFFFFFF);
        if (cur == 0x7FFFFFFF) return;  // the same in every wave and every split
    }
#pragma unroll
    for (int j = 0; j < kMaxStack; ++j) {
        if (j >= a.stack) break;
        const int next = min_of_16(id > cur ? id : 0x7FFFFFFF);
        if (next == 0x7FFFFFFF) {
            if (j == 0) return;
            break;
        }
        cur = next;
        list[j] = cur;
        if (id == cur) mine_at = j;
    }
    const uint32_t row_bytes = uint32_t(a.K) * 2u;
    const int steps = (a.K + kStepK - 1) / kStepK;
    const int s0 = int(int64_t(steps) * blockIdx.z / a.splits), s1 = int(int64_t(steps) * (blockIdx.z + 1) / a.splits);
    const auto x_rs = make_rsrc(a.X + row0 * a.K, uint32_t(have) * row_bytes);
    // a single adapter from its own 64-bit address (rows past the rank come as zeros), stacked ones by offsets into the
    // whole table (the host stacks where that is below 4 GiB)
    const bool stacked = RB == 1 && a.stack > 1;  // in one block (stack_of)
    const auto a_rs = make_rsrc(a.A + (stacked ? int64_t(0) : int64_t(list[0]) * a.rank * a.K),
                                (stacked ? uint32_t(a.adapters) : 1u) * uint32_t(a.rank) * row_bytes);
    // copy i of a block brings rows 4 i + lane / 16; X's rows of other adapters come as zeros
    constexpr uint32_t kNone = 0xFFFFFF00u;
    uint32_t x_off[4], a_off[RB][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + q;
        const uint32_t column = uint32_t(l16 ^ r) * 16u;
        x_off[i] = __shfl(mine_at, r) >= 0 ? uint32_t(r) * row_bytes + column : kNone;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            const int row = 16 * rb + r;
            if (!stacked) {
                a_off[rb][i] = row < a.rank ? uint32_t(row) * row_bytes + column : kNone;
            } else {
                const int j = row / a.rank;
                int e = -1;
#pragma unroll
                for (int k = 0; k < kMaxStack; ++k) e = j == k && k < a.stack ? list[k] : e;
                a_off[rb][i] = e >= 0 ? (uint32_t(e) * uint32_t(a.rank) + uint32_t(row - j * a.rank)) * row_bytes + column : kNone;
            }
        }
    }
    unsigned char* const at = lds[wave];
    int rd[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) rd[ks] = l16 * (kStepK * 2) + ((k_chunk(ks, q) ^ l16) << 4);
    f32x4_t acc[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) acc[rb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s = s0 + wave; s < s1; s += WAVES) {
        const uint32_t k0 = uint32_t(s) * (kStepK * 2u);
        const uint32_t left = row_bytes - k0;  // of a row; the last step may have half its columns
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = uint32_t(l16 ^ (4 * i + q)) * 16u < left;
            dma16(x_rs, at + i * 1024, in && x_off[i] != kNone ? x_off[i] + k0 : kNone, 0);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb)
                dma16(a_rs, at + (1 + rb) * kBlock + i * 1024, in && a_off[rb][i] != kNone ? a_off[rb][i] + k0 : kNone, 0);
        }
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const bf16x8_t xf = *reinterpret_cast<const bf16x8_t*>(at + rd[ks]);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb)
                acc[rb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    xf, *reinterpret_cast<const bf16x8_t*>(at + (1 + rb) * kBlock + rd[ks]), acc[rb], 0, 0, 0);
        }
        // the step's reads are done before the next copies may land
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        asm volatile("" ::: "memory");
    }
    // ---- the waves' sums, in wave order (each wave's in its own part of LDS: no copy is in flight) ----
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) reinterpret_cast<f32x4_t*>(at)[rb * 64 + lane] = acc[rb];
    __syncthreads();
    const int group = int(blockIdx.x) * int(gridDim.y) + int(blockIdx.y);
    constexpr int kSc1 = 16;  // through to the device-coherent level: other workgroups' caches are elsewhere
    const auto part_rs = make_rsrc(a.part + int64_t(group) * a.splits * (RB * 256), a.splits > 1 ? uint32_t(a.splits) * (RB * 1024u) : 0u);
    auto store = [&](int rb, f32x4_t v) __attribute__((always_inline)) {
        const int row = 16 * rb + l16, j = stacked ? row / a.rank : 0, r = row - j * a.rank;
        int adapter = -1;
#pragma unroll
        for (int k = 0; k < kMaxStack; ++k) adapter = j == k && k < a.stack ? list[k] : adapter;
        const bool in = adapter >= 0 && r < a.rank;
        const float alpha = in ? a.alpha[adapter] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int owner = __shfl(id, 4 * q + i);
            if (in && owner == adapter) {
                const float u = v[i] * alpha;
                const __bf16 hi = static_cast<__bf16>(u);
                const float h = static_cast<float>(hi);
                const bool fine = __builtin_fabsf(h) < __builtin_inff();  // an infinity's rest would be a NaN
                uint16_t* dst = a.u + (row0 + 4 * q + i) * (2 * a.rank) + r;
                dst[0] = __builtin_bit_cast(uint16_t, hi);
                dst[a.rank] = fine ? float_to_bf16_bits(u - h) : uint16_t(0);
            }
        }
    };
    for (int rb = wave; rb < RB; rb += WAVES) {
        f32x4_t v = reinterpret_cast<const f32x4_t*>(lds[0])[rb * 64 + lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            const f32x4_t o = reinterpret_cast<const f32x4_t*>(lds[w])[rb * 64 + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += o[i];
        }
        if (a.splits == 1)
            store(rb, v);
        else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), part_rs,
                                                   (uint32_t(blockIdx.z) * RB + uint32_t(rb)) * 1024u + uint32_t(lane) * 16u, 0, kSc1);
    }
    if (a.splits == 1) return;
    // ---- the splits' sums: the last to arrive adds them in order ----
    wait_vmcnt<0>();  // this one's sums are there before the arrival counts
    __syncthreads();
    if (threadIdx.x == 0)
        last_split = __hip_atomic_fetch_add(&a.counters[group], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == uint32_t(a.splits - 1);
    __syncthreads();
    if (!last_split) return;
    if (threadIdx.x == 0) __hip_atomic_store(&a.counters[group], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int rb = wave; rb < RB; rb += WAVES) {
        u32x4_t part[kMaxShrinkSplits];
#pragma unroll
        for (int z = 0; z < kMaxShrinkSplits; ++z)  // a split past the last reads as zeros
            part[z] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                      part_rs, (uint32_t(z) * RB + uint32_t(rb)) * 1024u + uint32_t(lane) * 16u, 0, kSc1));
        f32x4_t v = __builtin_bit_cast(f32x4_t, part[0]);
#pragma unroll
        for (int z = 1; z < kMaxShrinkSplits; ++z) {
            const f32x4_t o = __builtin_bit_cast(f32x4_t, part[z]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += o[i];
        }
        store(rb, v);
    }
}

int rank_blocks(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// Adapters that a workgroup stacks: as many as one block of 16 rows of A holds (X is then read by fewer workgroups and
// the block multiplied whole) where three workgroups for every four compute units are left.  K = 3072, first and second product,
// stacked / not: rank 8, 12 adapters, 400 rows (150 workgroups) 24.0 / 24.9 us, 512 (192) 23.8 / 24.7, 4608 50 / 66; 2 adapters,
// 2048 (128) 22.4 / 21.5, 4608 (288) 30.3 / 32.5.  A second block does not pay: rank 8, 12 adapters, 4608 rows 55 us with four;
// rank 16, 900 rows 33.3 / 29.9, 4608 70 / 65.
int stack_of(int64_t M, int64_t K, int64_t adapters, int rank) {
    const int64_t stack = 16 / rank < kMaxStack ? 16 / rank : kMaxStack;
    const int64_t among = adapters < 16 ? adapters : 16;  // in 16 rows
    if (stack < 2 || among < 2 || adapters * rank * K * 2 > (int64_t(1) << 32) - 1) return 1;
    return tiles_of(M, 16) * tiles_of(among, stack) < kComputeUnits * 3 / 4 ? 1 : int(stack);
}

int slots_of(int64_t adapters, int stack) { return int(tiles_of(adapters < 16 ? adapters : 16, stack)); }

// K is split where the row tiles leave compute units idle and a workgroup would read more than 256 KB (about
// 50 KB a microsecond arrive at a compute unit; the join costs 3 to 4 us): into pieces of 128 KB, and into
// kMaxParts pieces in all.
constexpr int kMaxParts = 1024;
int shrink_splits(int64_t M, int64_t K, int64_t adapters, int rank, int stack) {
    const int64_t tiles = tiles_of(M, 16), groups = tiles * slots_of(adapters, stack), bytes = (16 + int64_t(rank)) * K * 2;
    if (bytes <= 256 * 1024 || 2 * tiles > kComputeUnits || 2 * groups > kMaxParts) return 1;
    int64_t s = tiles_of(bytes, 128 * 1024);
    s = s < kComputeUnits / tiles ? s : kComputeUnits / tiles;
    s = s < kMaxParts / groups ? s : kMaxParts / groups;
    return int(s < kMaxShrinkSplits ? s : kMaxShrinkSplits);
}

}  // namespace

// The fp32 sums of the splits lie behind U.  Room for them is kept at every M, so that a workspace for
// some number of rows serves fewer as well.
size_t lora_u_bytes(int64_t M, int rank) { return (size_t(M) * size_t(rank) * 4u + 255u) & ~size_t(255); }
size_t lora_workspace_bytes(int64_t M, int rank) {
    const int64_t most = tiles_of(M, 16) * 16 * kMaxShrinkSplits, parts = most < kMaxParts ? most : kMaxParts;
    return kWorkspaceCounterBytes + lora_u_bytes(M, rank) + size_t(parts) * size_t(rank_blocks(rank < 32 ? 32 : rank)) * 1024u;
}

hipError_t launch_lora_shrink(ShrinkArgs a, void* workspace, hipStream_t stream) {
    unsigned char* const base = static_cast<unsigned char*>(workspace);
    a.counters = reinterpret_cast<uint32_t*>(base);
    a.u = reinterpret_cast<uint16_t*>(base + kWorkspaceCounterBytes);
    a.part = reinterpret_cast<float*>(base + kWorkspaceCounterBytes + lora_u_bytes(a.M, a.rank));
    a.stack = stack_of(a.M, a.K, a.adapters, a.rank);
    a.splits = shrink_splits(a.M, a.K, a.adapters, a.rank, a.stack);
    // a launch has at most 2^32 threads: more rows take several (not split, so without counters)
    const int64_t most = ((int64_t(1) << 23) - 1) * 16;
    for (int64_t left = a.M;; left -= most) {
        a.M = int(left < most ? left : most);
        const dim3 grid(unsigned(tiles_of(a.M, 16)), unsigned(slots_of(a.adapters, a.stack)), unsigned(a.splits));
        switch (rank_blocks(a.rank * a.stack)) {
            case 1: hipLaunchKernelGGL((lora_shrink_kernel<1, 8>), grid, dim3(512), 0, stream, a); break;
            case 2: hipLaunchKernelGGL((lora_shrink_kernel<2, 8>), grid, dim3(512), 0, stream, a); break;
            case 4: hipLaunchKernelGGL((lora_shrink_kernel<4, 4>), grid, dim3(256), 0, stream, a); break;
            default: hipLaunchKernelGGL((lora_shrink_kernel<8, 4>), grid, dim3(256), 0, stream, a); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || left <= most) return e;
        a.X += most * a.K;
        a.rows += most;
        a.u += most * 2 * a.rank;
    }
}

}  // namespace lowbit
