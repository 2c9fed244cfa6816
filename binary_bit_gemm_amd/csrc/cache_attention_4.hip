// Attention over a cache of 4-bit codes (cache_attention.h holds the kernel).
#include "cache_attention.h"

namespace lowbit {

hipError_t launch_cache_attention_4(const CacheAttnArgs& a, const CacheAttnPlan& plan, hipStream_t stream) {
    return a.cache.head_dim == 64 ? launch_cache_attention_as<64, 4>(a, plan, stream)
                                  : launch_cache_attention_as<128, 4>(a, plan, stream);
}

}  // namespace lowbit
