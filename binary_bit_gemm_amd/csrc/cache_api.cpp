// C-ABI of the decoding operators: the paged cache, attention over it, and matrix-vector products with affine 4-bit weights.
// As in lowbit_api.cpp, every check runs before any HIP call, and nothing here allocates or throws.
#include <hip/hip_runtime.h>

#include <limits>

#include "../../include/lowbit.h"
#include "host_checks.h"
#include "decode_internal.h"

namespace {

// The shape of a cache, and its arguments for the kernels; pointers are checked by cache_pointers().
int cache_shape(const lowbit_cache* c, lowbit::CacheArgs& a) {
    if (c == nullptr) return LOWBIT_E_INVALID;
    if (c->bits != 16 && c->bits != 8 && c->bits != 4) return LOWBIT_E_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return LOWBIT_E_UNSUPPORTED;
    int shift = 4;
    while (shift < 8 && (1 << shift) != c->page_size) ++shift;
    if ((1 << shift) != c->page_size) return LOWBIT_E_UNSUPPORTED;
    if (c->pages < 0 || c->kv_heads < 0) return LOWBIT_E_INVALID;
    if (c->kv_heads > kMaxHeads || c->pages > kMaxDim >> shift || c->pages * c->kv_heads > kMaxDim) return LOWBIT_E_UNSUPPORTED;
    a.k = static_cast<unsigned char*>(c->k);
    a.v = static_cast<unsigned char*>(c->v);
    a.k_scales = static_cast<unsigned char*>(c->k_scales);
    a.v_scales = static_cast<unsigned char*>(c->v_scales);
    a.pages = int(c->pages);
    a.page_shift = shift;
    a.heads = c->kv_heads;
    a.head_dim = c->head_dim;
    a.bits = c->bits;
    return LOWBIT_OK;
}

int cache_pointers(const lowbit::CacheArgs& a) {
    if (a.pages == 0) return LOWBIT_OK;  // nothing there to read or write
    if (a.k == nullptr || a.v == nullptr) return LOWBIT_E_INVALID;
    if (a.bits != 16 && (a.k_scales == nullptr || a.v_scales == nullptr)) return LOWBIT_E_INVALID;
    if (!aligned(a.k, 16) || !aligned(a.v, 16)) return LOWBIT_E_ALIGN;
    if (a.bits != 16 && (!aligned(a.k_scales, 16) || !aligned(a.v_scales, 16))) return LOWBIT_E_ALIGN;
    return LOWBIT_OK;
}

int cache_rows(const lowbit_cache* c, const void* k, const void* v, int64_t tokens, int64_t k_token, int64_t k_head, int64_t v_token,
               int64_t v_head, const int32_t* slots, bool write, void* stream) {
    lowbit::CacheArgs a{};
    int st = cache_shape(c, a);
    if (st != LOWBIT_OK) return st;
    if (tokens < 0) return LOWBIT_E_INVALID;
    if (tokens > kMaxDim) return LOWBIT_E_UNSUPPORTED;
    for (int64_t s : {k_token, k_head, v_token, v_head})
        if (!stride_ok(s)) return LOWBIT_E_INVALID;
    st = cache_pointers(a);
    if (st != LOWBIT_OK) return st;
    if (tokens == 0 || a.heads == 0 || a.pages == 0) return LOWBIT_OK;
    if (k == nullptr || v == nullptr || slots == nullptr) return LOWBIT_E_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return LOWBIT_E_ALIGN;
    if (!write && (!apart(tokens, k_token, a.heads, k_head, a.head_dim) || !apart(tokens, v_token, a.heads, v_head, a.head_dim)))
        return LOWBIT_E_INVALID;
    st = lowbit::device_check();
    if (st != LOWBIT_OK) return st;
    lowbit::CacheRows r{};
    r.k = static_cast<const uint16_t*>(k);
    r.v = static_cast<const uint16_t*>(v);
    if (!write) {
        r.k_out = static_cast<uint16_t*>(const_cast<void*>(k));
        r.v_out = static_cast<uint16_t*>(const_cast<void*>(v));
    }
    r.slots = slots;
    r.tokens = tokens;
    r.k_token = k_token;
    r.k_head = k_head;
    r.v_token = v_token;
    r.v_head = v_head;
    const hipError_t e = lowbit::launch_cache_rows(a, r, write, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? LOWBIT_OK : lowbit::hip_fail(e);
}

// The checks of lowbit_cache_attention that read no tensor pointer, and the launch arguments.
int attention_args(const lowbit_cache_attention_problem* p, lowbit::CacheAttnArgs& a) {
    if (p == nullptr) return LOWBIT_E_INVALID;
    const int st = cache_shape(&p->cache, a.cache);
    if (st != LOWBIT_OK) return st;
    if (p->batch < 0 || p->q_len < 0 || p->kv_len < 0 || p->q_heads < 0) return LOWBIT_E_INVALID;
    if (p->q_heads > kMaxHeads || p->batch > kMaxHeads) return LOWBIT_E_UNSUPPORTED;
    if (p->q_len > kMaxDim || p->kv_len > kMaxDim - 64) return LOWBIT_E_UNSUPPORTED;
    if (p->tree != nullptr && p->q_len > 64) return LOWBIT_E_UNSUPPORTED;
    const int heads = a.cache.heads;
    if (heads == 0 ? p->q_heads != 0 : p->q_heads % heads != 0) return LOWBIT_E_INVALID;
    if (!(p->scale > 0.f) || double(p->scale) * kLog2E > double(std::numeric_limits<float>::max())) return LOWBIT_E_INVALID;
    for (int64_t s : {p->q_batch, p->q_token, p->q_head, p->o_batch, p->o_token, p->o_head})
        if (!stride_ok(s)) return LOWBIT_E_INVALID;
    if (p->table_stride < 0 || p->table_stride > kMaxStride) return LOWBIT_E_INVALID;
    if (p->batch == 0 || p->q_len == 0 || p->q_heads == 0) return LOWBIT_OK;  // nothing to do: a.batch stays 0
    if (!apart3(p->batch, p->o_batch, p->q_len, p->o_token, p->q_heads, p->o_head, a.cache.head_dim)) return LOWBIT_E_INVALID;
    a.group = p->q_heads / heads;
    const int64_t rows = p->q_len * a.group;
    if (rows > kMaxDim - 64 || (rows + 15) / 16 * heads * p->batch > lowbit::kMaxGrid256) return LOWBIT_E_UNSUPPORTED;
    a.q = static_cast<const uint16_t*>(p->q);
    a.o = static_cast<uint16_t*>(p->o);
    a.table = p->page_table;
    a.lens = p->key_lens;
    a.q_lens = p->q_lens;
    a.tree = p->tree;
    a.q_batch = p->q_batch;
    a.q_token = p->q_token;
    a.q_head = p->q_head;
    a.o_batch = p->o_batch;
    a.o_token = p->o_token;
    a.o_head = p->o_head;
    a.table_stride = p->table_stride;
    a.batch = int(p->batch);
    a.q_len = int(p->q_len);
    a.kv_len = a.cache.pages > 0 ? int(p->kv_len) : 0;  // without pages there are no keys (and nothing to read)
    a.scale_log2 = float(double(p->scale) * kLog2E);
    return LOWBIT_OK;
}

}  // namespace

extern "C" {

int lowbit_cache_write(const lowbit_cache* cache, const void* k, const void* v, int64_t tokens, int64_t k_token, int64_t k_head,
                       int64_t v_token, int64_t v_head, const int32_t* slots, void* stream) {
    return cache_rows(cache, k, v, tokens, k_token, k_head, v_token, v_head, slots, true, stream);
}

int lowbit_cache_read(const lowbit_cache* cache, void* k, void* v, int64_t tokens, int64_t k_token, int64_t k_head, int64_t v_token,
                      int64_t v_head, const int32_t* slots, void* stream) {
    return cache_rows(cache, k, v, tokens, k_token, k_head, v_token, v_head, slots, false, stream);
}

size_t lowbit_cache_attention_workspace_size(const lowbit_cache_attention_problem* p) {
    lowbit::CacheAttnArgs a{};
    if (attention_args(p, a) != LOWBIT_OK || a.batch == 0) return 0;
    return lowbit::plan_cache_attention(a).bytes;
}

int lowbit_cache_attention(const lowbit_cache_attention_problem* p, void* workspace, size_t workspace_bytes, void* stream) {
    lowbit::CacheAttnArgs a{};
    int st = attention_args(p, a);
    if (st != LOWBIT_OK) return st;
    st = cache_pointers(a.cache);
    if (st != LOWBIT_OK) return st;
    if (a.batch == 0) return LOWBIT_OK;
    if (a.q == nullptr || a.o == nullptr || a.lens == nullptr || (a.kv_len > 0 && a.table == nullptr)) return LOWBIT_E_INVALID;
    if (!aligned(a.q, 16) || !aligned(a.o, 16) || !aligned(workspace, 16) || !aligned(a.tree, 8)) return LOWBIT_E_ALIGN;
    if (!aligned(a.table, 4) || !aligned(a.lens, 4) || !aligned(a.q_lens, 4)) return LOWBIT_E_ALIGN;
    st = lowbit::device_check();
    if (st != LOWBIT_OK) return st;
    lowbit::CacheAttnPlan plan = lowbit::plan_cache_attention(a);
    if (plan.bytes > 0 && (workspace == nullptr || workspace_bytes < plan.bytes)) plan = lowbit::plan_cache_attention(a, false);
    const hipError_t e = lowbit::launch_cache_attention(a, plan, workspace, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? LOWBIT_OK : lowbit::hip_fail(e);
}

int lowbit_gemv_affine(const void* X, const uint32_t* W, const void* S, const void* B, const void* residual, void* Y, int64_t M, int64_t N,
                       int64_t K, int g, int swiglu, void* stream) {
    const int64_t rows = swiglu && N >= 0 && N <= kMaxDim ? 2 * N : N;
    // N itself is checked with the others, as a multiple of 16; the weights' size with all their rows
    int st = lowbit_check_gemm_args(X, W, S, Y, M, N, K, g, 4);
    if (st != LOWBIT_OK) return st;
    if (rows > kMaxDim || rows * (K / 2) >= (int64_t(1) << 32)) return LOWBIT_E_UNSUPPORTED;
    if (M > lowbit::kGemvMaxRows || (g != 64 && g != 128)) return LOWBIT_E_UNSUPPORTED;
    if (M == 0 || N == 0) return LOWBIT_OK;
    if (K > 0 && B == nullptr) return LOWBIT_E_INVALID;
    if (!aligned(B, 16) || !aligned(residual, 16)) return LOWBIT_E_ALIGN;
    st = lowbit::device_check();
    if (st != LOWBIT_OK) return st;
    lowbit::GemvArgs a{};
    a.X = static_cast<const uint16_t*>(X);
    a.W = W;
    a.S = static_cast<const uint16_t*>(S);
    a.B = static_cast<const uint16_t*>(B);
    a.R = static_cast<const uint16_t*>(residual);
    a.Y = static_cast<uint16_t*>(Y);
    a.M = int(M);
    a.N = int(N);
    a.K = int(K);
    const hipError_t e = lowbit::launch_gemv_affine(a, g, swiglu != 0, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? LOWBIT_OK : lowbit::hip_fail(e);
}

}  // extern "C"
