// C-ABI of the operators around the packed linears: argument checks and launch.  As in lowbit_api.cpp,
// every check runs before any HIP call, and nothing here allocates or throws.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>
#include <limits>

#include "../../include/lowbit.h"
#include "lowbit_internal.h"

namespace {

bool aligned(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int kMaxHeads = 1 << 16;
constexpr double kLog2E = 1.4426950408889634074;

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride && s % 8 == 0; }

// Whether [tokens, heads] rows of `dim` elements at these strides lie apart (outputs).
bool apart(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
    if (tokens <= 1 && heads <= 1) return true;
    if (tokens <= 1) return head >= dim;
    if (heads <= 1) return token >= dim;
    return head <= token ? head >= dim && token >= (heads - 1) * head + dim
                         : token >= dim && head >= (tokens - 1) * token + dim;
}

// The same for [batch, tokens, heads] rows.
bool apart3(int64_t batch, int64_t batch_stride, int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
    if (batch == 0 || tokens == 0 || heads == 0) return true;
    int64_t n[3] = {batch, tokens, heads}, st[3] = {batch_stride, token, head};
    for (int i = 0; i < 2; ++i)  // by stride, smallest first
        for (int j = 0; j < 2 - i; ++j)
            if (st[j] > st[j + 1]) {
                const int64_t a = n[j], b = st[j];
                n[j] = n[j + 1];
                st[j] = st[j + 1];
                n[j + 1] = a;
                st[j + 1] = b;
            }
    int64_t span = dim;  // elements that the dimensions so far cover
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (st[i] < span) return false;
        span += (n[i] - 1) * st[i];
    }
    return true;
}

constexpr int64_t kMaxTokenStride = int64_t(1) << 24;  // 64 rows of keys within a 32-bit byte range

// The checks of lowbit_attention that read no tensor pointer, and the launch arguments.
int attention_args(const lowbit_attention_problem* p, lowbit::AttnArgs& a) {
    if (p == nullptr) return LOWBIT_E_INVALID;
    if (p->head_dim != 64 && p->head_dim != 128) return LOWBIT_E_UNSUPPORTED;
    if (p->batch < 0 || p->q_heads < 0 || p->kv_heads < 0 || p->q_len < 0 || p->kv_len < 0) return LOWBIT_E_INVALID;
    if (p->q_len > kMaxDim || p->kv_len > kMaxDim - 64) return LOWBIT_E_UNSUPPORTED;
    if (p->q_heads > kMaxHeads || p->batch > kMaxHeads) return LOWBIT_E_UNSUPPORTED;
    if (p->kv_heads == 0 ? p->q_heads != 0 : p->q_heads % p->kv_heads != 0) return LOWBIT_E_INVALID;
    // the kernels take scale * log2(e), which has to be finite as well
    if (!(p->scale > 0.f) || double(p->scale) * kLog2E > double(std::numeric_limits<float>::max())) return LOWBIT_E_INVALID;
    for (int64_t s : {p->q_batch, p->q_token, p->q_head, p->k_batch, p->k_token, p->k_head, p->v_batch, p->v_token,
                      p->v_head, p->o_batch, p->o_token, p->o_head})
        if (!stride_ok(s)) return LOWBIT_E_INVALID;
    if (p->mask_batch < 0 || p->mask_batch > kMaxStride) return LOWBIT_E_INVALID;
    if (p->batch == 0 || p->q_len == 0 || p->q_heads == 0) return LOWBIT_OK;  // nothing to do: a.rows stays 0
    if (p->kv_len > 1 && (p->k_token < p->head_dim || p->v_token < p->head_dim)) return LOWBIT_E_INVALID;
    if (p->k_token > kMaxTokenStride || p->v_token > kMaxTokenStride) return LOWBIT_E_UNSUPPORTED;
    if (!apart3(p->batch, p->o_batch, p->q_len, p->o_token, p->q_heads, p->o_head, p->head_dim)) return LOWBIT_E_INVALID;
    a.group = p->q_heads / p->kv_heads;
    const int64_t rows = int64_t(p->q_len) * a.group;
    if (rows > kMaxDim - 128 || (rows + 127) / 128 * p->kv_heads * p->batch > lowbit::kMaxGrid256) return LOWBIT_E_UNSUPPORTED;
    a.q_batch = p->q_batch;
    a.q_token = p->q_token;
    a.q_head = p->q_head;
    a.k_batch = p->k_batch;
    a.k_token = p->kv_len > 1 ? p->k_token : p->head_dim;
    a.k_head = p->k_head;
    a.v_batch = p->v_batch;
    a.v_token = p->kv_len > 1 ? p->v_token : p->head_dim;
    a.v_head = p->v_head;
    a.o_batch = p->o_batch;
    a.o_token = p->o_token;
    a.o_head = p->o_head;
    a.mask_batch = p->mask_batch;
    a.batch = int(p->batch);
    a.kv_heads = p->kv_heads;
    a.rows = int(rows);
    a.kv_len = int(p->kv_len);
    a.causal = p->causal != 0;
    a.scale_log2 = float(double(p->scale) * kLog2E);
    a.q = static_cast<const uint16_t*>(p->q);
    a.k = static_cast<const uint16_t*>(p->k);
    a.v = static_cast<const uint16_t*>(p->v);
    a.o = static_cast<uint16_t*>(p->o);
    a.mask = p->key_mask;
    a.lens = p->key_lens;
    a.start = p->q_start;
    return LOWBIT_OK;
}

constexpr int64_t kMaxAdapters = 1 << 16;

bool lora_rank_ok(int64_t rank) { return rank >= 8 && rank <= 128 && rank % 8 == 0; }

}  // namespace

extern "C" {

size_t lowbit_lora_workspace_size(int64_t M, int rank) {
    if (M <= 0 || M > kMaxDim || !lora_rank_ok(rank)) return 0;
    return lowbit::lora_workspace_bytes(M, rank);
}

size_t lowbit_lora_split_workspace_size(int64_t M, int64_t N, int64_t K, int g, int bits, int rank) {
    if (M <= 0 || N <= 0 || K <= 0 || !lora_rank_ok(rank) ||
        lowbit_check_gemm_args(nullptr, nullptr, nullptr, nullptr, 0, N, K, g, bits) != LOWBIT_OK || M > kMaxDim ||
        !lowbit::tile16_supported(g, bits))
        return 0;
    const lowbit::GemmProblem p{nullptr, nullptr, nullptr, nullptr, int(M), int(N), int(K)};
    const bool few = lowbit::use_skinny(M, N, K, g, bits);  // those kernels split K inside a workgroup
    return lowbit::lora_workspace_bytes(M, rank) + (few ? 0 : lowbit::lora_split_bytes(p, g, bits));
}

int lowbit_gemm_lora(const void* X, const uint32_t* W, const void* S, void* Y, int64_t M, int64_t N, int64_t K, int g,
                     int bits, const void* A, const void* B, const float* alpha, const int32_t* rows, int64_t adapters,
                     int rank, void* workspace, size_t workspace_bytes, void* stream) {
    int st = lowbit_check_gemm_args(X, W, S, Y, M, N, K, g, bits);
    if (st != LOWBIT_OK) return st;
    if (!lora_rank_ok(rank) || adapters > kMaxAdapters) return LOWBIT_E_UNSUPPORTED;
    if (adapters < 0) return LOWBIT_E_INVALID;
    if (!lowbit::tile16_supported(g, bits)) return LOWBIT_E_UNSUPPORTED;
    if (N * int64_t(rank) * 2 > (int64_t(1) << 32) - 1) return LOWBIT_E_UNSUPPORTED;
    if (M * N == 0) return LOWBIT_OK;
    // no adapter, or an empty sum: the plain product
    if (adapters == 0 || K == 0) return lowbit_gemm(X, W, S, Y, M, N, K, g, bits, stream);
    if (A == nullptr || B == nullptr || alpha == nullptr || rows == nullptr) return LOWBIT_E_INVALID;
    if (workspace == nullptr || workspace_bytes < lowbit_lora_workspace_size(M, rank)) return LOWBIT_E_INVALID;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(workspace, 16) || !aligned(alpha, 4) || !aligned(rows, 4))
        return LOWBIT_E_ALIGN;
    st = lowbit::device_check();
    if (st != LOWBIT_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    lowbit::ShrinkArgs sh{};
    sh.X = static_cast<const uint16_t*>(X);
    sh.A = static_cast<const uint16_t*>(A);
    sh.alpha = alpha;
    sh.rows = rows;
    sh.M = int(M);
    sh.K = int(K);
    sh.adapters = int(adapters);
    sh.rank = rank;
    hipError_t e = lowbit::launch_lora_shrink(sh, workspace, s);
    if (e != hipSuccess) return lowbit::hip_fail(e);
    const lowbit::LoraArgs la{lowbit::lora_u(workspace), static_cast<const uint16_t*>(B), rows, int(adapters), rank};
    const lowbit::GemmProblem p{static_cast<const uint16_t*>(X), W, static_cast<const uint16_t*>(S),
                                static_cast<uint16_t*>(Y), int(M), int(N), int(K)};
    // few rows: the kernels that lowbit_gemm takes for them, where they cover the shape
    e = hipErrorNotSupported;
    if (bits == 2 && M <= 16 && N / 16 >= 512) e = lowbit::launch_gemm_resident_epilogue(p, g, lowbit::kEpiLora, s, &la);
    if (e == hipErrorNotSupported && lowbit::use_skinny(M, N, K, g, bits)) e = lowbit::launch_gemm_skinny_group(&p, 1, g, bits, s, &la);
    if (e == hipErrorNotSupported) {
        const size_t least = lowbit::lora_workspace_bytes(M, rank), sums = lowbit::lora_split_bytes(p, g, bits);
        void* const at = sums > 0 && workspace_bytes >= least + sums ? static_cast<unsigned char*>(workspace) + least : nullptr;
        e = lowbit::launch_gemm_tile16_lora(p, g, bits, la, workspace, at, s);
    }
    return e == hipSuccess ? LOWBIT_OK : lowbit::hip_fail(e);
}

size_t lowbit_attention_workspace_size(const lowbit_attention_problem* p) {
    lowbit::AttnArgs a{};
    if (attention_args(p, a) != LOWBIT_OK || a.batch == 0 || a.rows == 0) return 0;
    return lowbit::plan_attention(a, p->head_dim).bytes;
}

int lowbit_attention(const lowbit_attention_problem* p, void* workspace, size_t workspace_bytes, void* stream) {
    lowbit::AttnArgs a{};
    int st = attention_args(p, a);
    if (st != LOWBIT_OK) return st;
    if (a.batch == 0 || a.rows == 0) return LOWBIT_OK;
    if (a.q == nullptr || a.o == nullptr) return LOWBIT_E_INVALID;
    if (a.kv_len > 0 && (a.k == nullptr || a.v == nullptr)) return LOWBIT_E_INVALID;
    for (const void* ptr : {p->q, p->k, p->v, static_cast<const void*>(p->o), static_cast<const void*>(workspace)})
        if (!aligned(ptr, 16)) return LOWBIT_E_ALIGN;
    if (!aligned(p->key_lens, 4) || !aligned(p->q_start, 4)) return LOWBIT_E_ALIGN;
    st = lowbit::device_check();
    if (st != LOWBIT_OK) return st;
    lowbit::AttnPlan plan = lowbit::plan_attention(a, p->head_dim);
    if (plan.bytes > 0 && (workspace == nullptr || workspace_bytes < plan.bytes))
        plan = lowbit::plan_attention(a, p->head_dim, false);
    const hipError_t e = lowbit::launch_attention(a, p->head_dim, plan, workspace, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? LOWBIT_OK : lowbit::hip_fail(e);
}

int lowbit_qk_norm_rope(const lowbit_qk_problem* p, void* stream) {
    if (p == nullptr) return LOWBIT_E_INVALID;
    const int D = p->head_dim;
    if (D != 32 && D != 64 && D != 128 && D != 256) return LOWBIT_E_UNSUPPORTED;
    if (p->axes < 0 || p->axes > 4) return LOWBIT_E_UNSUPPORTED;
    if (p->tokens < 0 || p->tokens > kMaxDim || p->q_heads < 0 || p->k_heads < 0) return LOWBIT_E_INVALID;
    if (p->q_heads > kMaxHeads || p->k_heads > kMaxHeads) return LOWBIT_E_UNSUPPORTED;
    lowbit::QkArgs a{};
    int rot = 0;
    for (int i = 0; i < p->axes; ++i) {
        const int d = p->axis_dims[i];
        if (d <= 0 || d % 2 != 0 || d > D) return LOWBIT_E_INVALID;
        rot += d;
        a.axis_end[i] = rot / 2;
    }
    if (rot % 16 != 0 || rot > D) return LOWBIT_E_INVALID;
    for (int i = p->axes; i < 4; ++i) a.axis_end[i] = rot / 2;
    if (!(p->eps >= 0.f) || std::isinf(p->eps)) return LOWBIT_E_INVALID;
    for (int64_t s : {p->q_token, p->q_head, p->k_token, p->k_head, p->q_out_token, p->q_out_head, p->k_out_token,
                      p->k_out_head})
        if (!stride_ok(s)) return LOWBIT_E_INVALID;
    if (p->tokens == 0 || p->q_heads + p->k_heads == 0) return LOWBIT_OK;
    if (p->q_heads > 0 && (p->q == nullptr || p->q_out == nullptr)) return LOWBIT_E_INVALID;
    if (p->k_heads > 0 && (p->k == nullptr || p->k_out == nullptr)) return LOWBIT_E_INVALID;
    if (p->axes > 0 && (p->positions == nullptr || p->freqs == nullptr)) return LOWBIT_E_INVALID;
    if (!apart(p->tokens, p->q_out_token, p->q_heads, p->q_out_head, D) ||
        !apart(p->tokens, p->k_out_token, p->k_heads, p->k_out_head, D))
        return LOWBIT_E_INVALID;
    // in place: the same element order (a stride along a dimension of one element says nothing)
    auto moved = [&](const void* in, const void* out, int heads, int64_t it, int64_t ih, int64_t ot, int64_t oh) {
        return heads > 0 && in == out && ((p->tokens > 1 && it != ot) || (heads > 1 && ih != oh));
    };
    if (moved(p->q, p->q_out, p->q_heads, p->q_token, p->q_head, p->q_out_token, p->q_out_head) ||
        moved(p->k, p->k_out, p->k_heads, p->k_token, p->k_head, p->k_out_token, p->k_out_head))
        return LOWBIT_E_INVALID;
    for (const void* ptr : {p->q, p->k, static_cast<const void*>(p->q_out), static_cast<const void*>(p->k_out),
                            p->q_weight, p->k_weight})
        if (!aligned(ptr, 16)) return LOWBIT_E_ALIGN;
    if (!aligned(p->positions, 4) || !aligned(p->freqs, 4)) return LOWBIT_E_ALIGN;
    const int st = lowbit::device_check();
    if (st != LOWBIT_OK) return st;
    a.q = static_cast<const uint16_t*>(p->q);
    a.k = static_cast<const uint16_t*>(p->k);
    a.q_out = static_cast<uint16_t*>(p->q_out);
    a.k_out = static_cast<uint16_t*>(p->k_out);
    a.q_weight = static_cast<const uint16_t*>(p->q_weight);
    a.k_weight = static_cast<const uint16_t*>(p->k_weight);
    a.positions = p->positions;
    a.freqs = p->freqs;
    a.tokens = p->tokens;
    a.q_token = p->q_token;
    a.q_head = p->q_head;
    a.k_token = p->k_token;
    a.k_head = p->k_head;
    a.qo_token = p->q_out_token;
    a.qo_head = p->q_out_head;
    a.ko_token = p->k_out_token;
    a.ko_head = p->k_out_head;
    a.q_heads = p->q_heads;
    a.k_heads = p->k_heads;
    a.axes = p->axes;
    a.rot = rot;
    a.eps = p->eps;
    const hipError_t e = lowbit::launch_qk_norm_rope(a, D, p->interleaved != 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? LOWBIT_OK : lowbit::hip_fail(e);
}

}  // extern "C"
