// cache_attention_fp16.hip -- the cached attention's kernels for float16 queries and a cache
// of their type (cache_attention.hpp).
#define AR_ATTEND_FAMILY
#include "cache_attention.hpp"

namespace ar {

template hipError_t launch_attend<Fp16, false>(const CacheAttentionArgs &, bool, int, hipStream_t);

}  // namespace ar
