// cache_attention_fp16_eight.hip -- the cached attention's kernels for float16 queries, a cache
// in 8 bits with scales and up to 16 query heads to a key-value head
// (cache_attention.hpp).
#define AR_ATTEND_FAMILY
#include "cache_attention.hpp"

namespace ar {

template hipError_t launch_attend<Fp16, true, 1>(const CacheAttentionArgs &, bool, int, hipStream_t);

}  // namespace ar
