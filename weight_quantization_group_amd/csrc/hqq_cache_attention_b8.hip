// hqq_cache_attention_b8.hip -- the cache's attention at 8 bits.
#include "hqq_cache_attention.h"

namespace hqq {

hipError_t launch_cache_attention_b8(int dim, int group_size, const CacheAttentionArgs &a, hipStream_t s)
{
    return a.bf16 ? launch_cache_attention<8, true>(dim, group_size, a, s)
                  : launch_cache_attention<8, false>(dim, group_size, a, s);
}

}  // namespace hqq
