// cache_attention_bf16.hip -- the cached attention's kernels for bfloat16 queries, a cache
// of their type and up to 16 query heads to a key-value head
// (cache_attention.hpp).
#define AR_ATTEND_FAMILY
#include "cache_attention.hpp"

namespace ar {

template hipError_t launch_attend<Bf16, false, 1>(const CacheAttentionArgs &, bool, int, hipStream_t);

}  // namespace ar
