// cache_attention_fp32_eight_wide.hip -- the cached attention's kernels for float32 queries, a cache
// in 8 bits with scales and more than 16 query heads to a key-value head
// (cache_attention.hpp).
#define AR_ATTEND_FAMILY
#include "cache_attention.hpp"

namespace ar {

template hipError_t launch_attend<Fp32, true, 2>(const CacheAttentionArgs &, bool, int, hipStream_t);

}  // namespace ar
