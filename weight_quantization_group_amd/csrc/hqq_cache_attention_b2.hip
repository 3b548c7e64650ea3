// hqq_cache_attention_b2.hip -- the cache's attention at 2 bits.
#include "hqq_cache_attention.h"

namespace hqq {

hipError_t launch_cache_attention_b2(int dim, int group_size, const CacheAttentionArgs &a, hipStream_t s)
{
    return launch_cache_attention<2>(dim, group_size, a, s);
}

}  // namespace hqq
