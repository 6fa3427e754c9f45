// cache_attention_fp16_wide.hip -- the cached attention's kernels for float16 queries, a cache
// of their type and more than 16 query heads to a key-value head
// (cache_attention.hpp).
#define AR_ATTEND_FAMILY
#include "cache_attention.hpp"

namespace ar {

template hipError_t launch_attend<Fp16, false, 2>(const CacheAttentionArgs &, bool, int, hipStream_t);

}  // namespace ar
