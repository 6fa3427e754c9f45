// cache_attention.hip -- the choice among the cached attention's kernel families
// (cache_attention.hpp) and the size of its workspace.
#include "cache_attention.hpp"

namespace ar {

uint64_t cache_attention_workspace(uint32_t dim, int cu_count)
{
    const uint64_t most = attend_most(2, cu_count);
    return most * 16u + most * 2u * attend_slot(padded_dim(dim)) * sizeof(float);
}

hipError_t launch_cache_attention(const CacheAttentionArgs &args, int dtype, bool eight,
                                  bool eight_out, int cu_count, hipStream_t stream)
{
    switch (dtype) {
    case kBf16:
        return eight ? launch_attend<Bf16, true>(args, eight_out, cu_count, stream)
                     : launch_attend<Bf16, false>(args, eight_out, cu_count, stream);
    case kFp16:
        return eight ? launch_attend<Fp16, true>(args, eight_out, cu_count, stream)
                     : launch_attend<Fp16, false>(args, eight_out, cu_count, stream);
    default:
        return eight ? launch_attend<Fp32, true>(args, eight_out, cu_count, stream)
                     : launch_attend<Fp32, false>(args, eight_out, cu_count, stream);
    }
}

}  // namespace ar
