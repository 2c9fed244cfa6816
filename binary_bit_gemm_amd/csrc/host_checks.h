// Argument checks that the entry points share (host code).
#pragma once

#include <stdint.h>

namespace {

inline bool aligned(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int kMaxHeads = 1 << 16;
constexpr double kLog2E = 1.4426950408889634074;

inline bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride && s % 8 == 0; }

// Whether [tokens, heads] rows of `dim` elements at these strides lie apart (outputs).
inline bool apart(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
    if (tokens <= 1 && heads <= 1) return true;
    if (tokens <= 1) return head >= dim;
    if (heads <= 1) return token >= dim;
    return head <= token ? head >= dim && token >= (heads - 1) * head + dim
                         : token >= dim && head >= (tokens - 1) * token + dim;
}

// The same for [batch, tokens, heads] rows.
inline bool apart3(int64_t batch, int64_t batch_stride, int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
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

}  // namespace
